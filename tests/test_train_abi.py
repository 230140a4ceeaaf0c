"""Refusals of the training operators and the AdamW table, on the CPU (no device is touched: every
call here returns before a launch), and the same entry points under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import fp8_block_scaled_e4m3_amd as dg

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
BF16, F16, F32 = 1, 2, 0
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, dg.DG_ERR_INVALID_ARG, dg.DG_ERR_UNSUPPORTED, dg.DG_ERR_MISALIGNED
A, B, D, OFF = 0x10000, 0x20000, 0x30000, 0x40000     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return dg.load_library()


def weights_call(lib, name, **change):
    args = dict(a=A, lda=128, b=B, d=D, ldd=128, offsets=OFF, m=10, n=64, k=128, g=4, dtype=BF16, workspace=None, bytes=0, stream=None)
    if name.endswith("nn"):
        args.update(lda=64, ldd=128)
    args.update(change)
    return getattr(lib, name)(*args.values())


WEIGHTS = ["dg_m_grouped_gemm_ragged_nt", "dg_m_grouped_gemm_ragged_nn"]


@pytest.mark.parametrize("name", WEIGHTS)
@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(n=-8), INVALID), (dict(k=-8), INVALID), (dict(g=0), INVALID),
    (dict(dtype=F32), INVALID), (dict(dtype=7), INVALID), (dict(lda=56), INVALID), (dict(ldd=56), INVALID),
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(d=None), INVALID), (dict(offsets=None), INVALID),
    (dict(n=60), UNSUPPORTED), (dict(k=100), UNSUPPORTED), (dict(g=1025), UNSUPPORTED),
    (dict(lda=1 << 21), UNSUPPORTED), (dict(ldd=1 << 21), UNSUPPORTED), (dict(lda=1 << 40), UNSUPPORTED),
    (dict(a=A + 8), MISALIGNED), (dict(b=B + 2), MISALIGNED), (dict(d=D + 4), MISALIGNED), (dict(lda=132), MISALIGNED),
    (dict(ldd=1028), MISALIGNED), (dict(offsets=OFF + 2), MISALIGNED),
    (dict(bytes=-1), INVALID), (dict(bytes=64), INVALID), (dict(workspace=0x50008, bytes=64), MISALIGNED),
    (dict(m=(1 << 30) + 1), UNSUPPORTED), (dict(m=0), OK), (dict(m=0, a=None), OK)])
def test_products_with_weights_refuse(lib, name, change, status):
    assert weights_call(lib, name, **change) == status


def test_empty_extents(lib):
    nt, nn = WEIGHTS
    assert weights_call(lib, nt, n=0) == OK and weights_call(lib, nn, k=0) == OK          # nothing to write
    assert weights_call(lib, nt, k=0) == UNSUPPORTED and weights_call(lib, nn, n=0) == UNSUPPORTED


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(g=0), INVALID), (dict(dtype=F32), INVALID), (dict(d_dtype=F16), INVALID),
    (dict(d_dtype=9), INVALID), (dict(accumulate=2), INVALID), (dict(lda=56), INVALID), (dict(ldb=120), INVALID),
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(d=None), INVALID), (dict(offsets=None), INVALID),
    (dict(n=4), UNSUPPORTED), (dict(k=4), UNSUPPORTED), (dict(g=5000), UNSUPPORTED), (dict(ldb=1 << 21), UNSUPPORTED),
    (dict(a=A + 2), MISALIGNED), (dict(b=B + 8), MISALIGNED), (dict(d=D + 8), MISALIGNED), (dict(ldb=130), MISALIGNED),
    (dict(bytes=-1), INVALID), (dict(bytes=64), INVALID), (dict(workspace=0x50004, bytes=64), MISALIGNED),
    (dict(n=0), OK), (dict(k=0), OK), (dict(m=0, accumulate=1), OK), (dict(m=0, accumulate=1, a=None, b=None), OK)])
def test_weight_gradient_refuses(lib, change, status):
    args = dict(a=A, lda=64, b=B, ldb=128, d=D, offsets=OFF, m=10, n=64, k=128, g=4, dtype=BF16, d_dtype=BF16,
                accumulate=0, workspace=None, bytes=0, stream=None)
    args.update(change)
    assert lib.dg_k_grouped_gemm_ragged_tn(*args.values()) == status


def test_ragged_tile_hooks(lib):
    tiles = dg.dg_ragged_tile_info()
    assert (128, 128) in tiles and (256, 256) in tiles and len(set(tiles)) == len(tiles)
    for t in tiles + [(128, 128, 4), (0, 0)]:
        dg.dg_set_ragged_tile(*t)
    assert lib.dg_set_ragged_tile(17, 32, 0) == INVALID and lib.dg_set_ragged_tile(128, 128, 33) == INVALID
    assert lib.dg_set_ragged_tile(128, 128, -1) == INVALID and lib.dg_ragged_tile_info(0, None) == INVALID
    assert lib.dg_ragged_tile_info(-1, (ctypes.c_int * 2)()) == INVALID


@pytest.mark.parametrize("args,status", [
    ((3, 10, 64, 64, 1, BF16, BF16), INVALID), ((-1, 10, 64, 64, 1, BF16, BF16), INVALID), ((0, -1, 64, 64, 1, BF16, BF16), INVALID),
    ((0, 10, 60, 64, 1, BF16, BF16), UNSUPPORTED), ((0, 10, 64, 64, 1, F32, F32), INVALID), ((0, 10, 64, 64, 1, BF16, F32), INVALID),
    ((2, 10, 64, 64, 1, BF16, F16), INVALID), ((2, 0, 64, 64, 1, BF16, F32), 0), ((1, 10, 0, 64, 1, F16, F16), 0)])
def test_workspace_bytes(lib, args, status):
    assert lib.dg_ragged_workspace_bytes(*args) == status


def tensor(**change):
    t = dg._AdamwTensor(param=0x1000, grad=0x2000, exp_avg=0x3000, exp_avg_sq=0x4000, numel=5000, param_dtype=F32,
                        grad_dtype=BF16, copy_dtype=0, state_format=dg.DG_STATE_F32)
    for key, value in change.items():
        setattr(t, key, value)
    return t


FP8 = dict(state_format=dg.DG_STATE_E4M3, exp_avg_scale=0x5000, exp_avg_sq_scale=0x6000)


@pytest.mark.parametrize("change,status", [
    (dict(numel=-1), INVALID), (dict(param=None), INVALID), (dict(grad=None), INVALID), (dict(exp_avg=None), INVALID),
    (dict(exp_avg_sq=None), INVALID), (dict(param_dtype=F16), INVALID), (dict(grad_dtype=5), INVALID),
    (dict(copy=0x7000, copy_dtype=F32), INVALID), (dict(state_format=2), INVALID),
    (dict(FP8, exp_avg_scale=None), INVALID), (dict(FP8, exp_avg_sq_scale=None), INVALID),
    (dict(numel=1 << 43), UNSUPPORTED), (dict(numel=(1 << 63) - 1), UNSUPPORTED),
    (dict(param=0x1008), MISALIGNED), (dict(grad=0x2002), MISALIGNED), (dict(copy=0x7004, copy_dtype=BF16), MISALIGNED),
    (dict(exp_avg=0x3008), MISALIGNED), (dict(FP8, exp_avg=0x3004), MISALIGNED), (dict(FP8, exp_avg_scale=0x5002), MISALIGNED)])
def test_adamw_plan_refuses(lib, change, status):
    tensors = (dg._AdamwTensor * 2)(tensor(), tensor(**change))
    assert lib.dg_adamw_plan_bytes(tensors, 2) == status
    buf = ctypes.create_string_buffer(1 << 16)
    assert lib.dg_adamw_plan(tensors, 2, buf, 1 << 16) == status


def test_adamw_table(lib):
    """An entry of 72 bytes a tensor, then the tensor of each chunk of 2048 elements."""
    sizes = [1, 2048, 0, 2049, 10000]
    tensors = (dg._AdamwTensor * 5)(*[tensor(numel=s) for s in sizes])
    chunks = [0, 1, 3, 3, 4, 4, 4, 4, 4]
    nbytes = lib.dg_adamw_plan_bytes(tensors, 5)
    assert nbytes == 5 * 72 + 4 * len(chunks)
    buf = ctypes.create_string_buffer(nbytes)
    assert lib.dg_adamw_plan(tensors, 5, buf, nbytes - 4) == INVALID
    assert lib.dg_adamw_plan(tensors, 5, None, nbytes) == INVALID
    assert lib.dg_adamw_plan(tensors, 5, buf, nbytes) == OK
    assert np.frombuffer(buf.raw[5 * 72:], np.int32).tolist() == chunks
    first = [np.frombuffer(buf.raw[i * 72 + 64:i * 72 + 68], np.int32)[0] for i in range(5)]
    assert first == [0, 1, 2, 2, 4]
    assert lib.dg_adamw_plan_bytes(None, 0) == 0 and lib.dg_adamw_plan(None, 0, None, 0) == OK
    assert lib.dg_adamw_plan_bytes(None, 1) == INVALID and lib.dg_adamw_plan_bytes(tensors, -1) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(step=0), INVALID), (dict(count=-1), INVALID), (dict(bytes=71), INVALID), (dict(bytes=74), INVALID),
    (dict(beta1=1.0), INVALID), (dict(beta1=-0.1), INVALID), (dict(beta2=1.0), INVALID), (dict(beta2=float("nan")), INVALID),
    (dict(eps=-1e-9), INVALID), (dict(eps=float("inf")), INVALID), (dict(lr=float("nan")), INVALID),
    (dict(wd=float("inf")), INVALID), (dict(table=None), INVALID), (dict(table=0x1004), MISALIGNED),
    (dict(grad_scale=0x2002), MISALIGNED), (dict(count=0, bytes=0), OK), (dict(bytes=72), OK)])
def test_adamw_step_refuses(lib, change, status):
    args = dict(table=0x1000, count=1, bytes=76, step=1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1, grad_scale=None,
                stream=None)
    args.update(change)
    assert lib.dg_adamw_step(*args.values()) == status


def test_binding_refuses_before_the_library():
    import torch
    a, b, off = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(2, 8, 16, dtype=torch.bfloat16), torch.zeros(3)
    with pytest.raises(ValueError):            # CPU tensors
        dg.dg_m_grouped_gemm_ragged_nt(a, b, torch.zeros(4, 8, dtype=torch.bfloat16), off)
    with pytest.raises(ValueError):
        dg.dg_adamw_plan([a], [a], [a], [a])
    with pytest.raises(ValueError):            # one moment's scales without the other's
        dg.dg_adamw_plan([a], [a], [a], [a], exp_avg_scales=[a])
    with pytest.raises(ValueError):
        dg.dg_adamw_plan([a], [], [a], [a])


def test_entry_points_under_sanitizers(tmp_path):
    """dg_train_api.cpp unchanged, with recording stand-ins for the kernels (host_models/train_host_check.cpp)."""
    include = "/opt/rocm/include"
    if not shutil.which("g++") or not os.path.isdir(os.path.join(include, "hip")):
        pytest.skip("needs g++ and the HIP headers")
    exe = str(tmp_path / "train_host_check")
    subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-I" + include,
                    os.path.join(ROOT, "fp8_block_scaled_e4m3_amd", "csrc", "dg_train_api.cpp"),
                    os.path.join(HERE, "host_models", "train_host_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "0 failures" in r.stdout, r.stdout + r.stderr[-4000:]
