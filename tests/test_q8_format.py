"""CPU checks of the 8-bit cache: the oracle's format against torch's e4m3 and closed forms, and
the host validation of its entry points (which fails before anything is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_attention_cb_gb300 as cb
from oracle import kv_q8
from paged_kv_attention_cb_gb300 import build as cbbuild

FAKE = 0x100000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    cbbuild.build()
    return cb.lib()


def test_grid_is_torchs_e4m3():
    c = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c, kv_q8.e4m3_values())


def test_rounding_is_torchs():
    x = np.random.default_rng(0).normal(size=20000) * np.exp2(np.random.default_rng(1).integers(-12, 8, 20000))
    x = np.concatenate([x, kv_q8.e4m3_values(), (kv_q8.e4m3_values()[1:] + kv_q8.e4m3_values()[:-1]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, kv_q8.round_e4m3(x))


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.0 * 1.0001, 1), (449.0, 1), (896.0, 1), (1.75, -8),
                                   (1.7500001, -7), (1.0, -8), (0.0, 0), (2.0 ** -149, -126),
                                   (3.4e38, 120)])
def test_scale_of_a_row(top, e):
    x = np.array([[0.0, np.float32(top), -np.float32(top) / 3, 0.0]])
    y, got = kv_q8.quantise_rows(x)
    assert got[0] == e
    assert np.abs(y).max() <= 448


def test_round_trip_of_codes():
    x = np.random.default_rng(3).normal(size=(50, 64)) * 7
    x[3] = 0
    y, e = kv_q8.quantise_rows(x)
    c, s = kv_q8.codes(y, e)
    assert np.array_equal(kv_q8.values(c, s), y * np.exp2(e.astype(float))[:, None])
    # half a step of 3 fraction bits, or half the smallest step below the normal range
    tol = np.maximum(np.abs(x) * 2.0 ** -4, np.exp2(e.astype(float))[:, None] * 2.0 ** -10)
    assert (np.abs(kv_q8.values(c, s) - x) <= tol).all()


def test_special_values():
    y, e = kv_q8.quantise_rows(np.array([[np.inf, -np.inf, np.nan, 3.0]]))
    assert e[0] == -7 and y[0, 0] == 448 and y[0, 1] == -448 and np.isnan(y[0, 2])


# ------------------------------------------------------------------ refusals


def rows_call(lib, name, *, k=FAKE, cache=FAKE, scale=FAKE, slots=FAKE, T=4, NB=10, BS=16, H=2, D=64,
              dtype=1):
    if name == "cb_write_kv_q8":
        return lib.cb_write_kv_q8(k, FAKE, cache, FAKE, scale, FAKE, slots, T, NB, BS, H, D, dtype,
                                  None, None)
    return lib.cb_read_kv_q8(cache, FAKE, scale, FAKE, slots, k, FAKE, T, NB, BS, H, D, dtype, None,
                             None)


@pytest.mark.parametrize("name", ["cb_write_kv_q8", "cb_read_kv_q8"])
@pytest.mark.parametrize("kwargs,status", [
    (dict(D=96), 3), (dict(D=256), 3), (dict(dtype=2), 1), (dict(T=-1), 1), (dict(NB=0), 1),
    (dict(BS=0), 1), (dict(H=0), 1), (dict(k=None), 1), (dict(cache=None), 1),
    (dict(scale=None), 1), (dict(slots=None), 1), (dict(k=FAKE + 8), 1), (dict(cache=FAKE + 4), 1),
    (dict(scale=FAKE + 1), 1), (dict(T=0, k=None), 0),
])
def test_rows_refusals(lib, name, kwargs, status):
    assert rows_call(lib, name, **kwargs) == status
    assert status == 0 or lib.cb_last_error_message()


def step_call(lib, qsl, seq, *, T=None, NB=40, BS=16, Hq=4, Hkv=2, D=64, dtype=1, stride=None,
              ws_bytes=None, chunk=0, workspace=FAKE, out=FAKE, scale_ptr=FAKE, k_new=None, v_new=None,
              mirrors=True):
    qsl = np.ascontiguousarray(qsl, np.int32)
    seq = np.ascontiguousarray(seq, np.int32)
    R = len(seq)
    T = int(qsl[-1]) if T is None else T
    if stride is None:
        stride = max(1, int(max((seq + BS - 1) // BS))) if R else 1
    if ws_bytes is None:
        ws_bytes = lib.cb_workspace_size_q8(R, T, Hq, Hkv, D, BS, chunk)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    return lib.cb_paged_attention_q8(out, FAKE, FAKE, FAKE, scale_ptr, FAKE, k_new, v_new, None, FAKE, FAKE,
                                     FAKE, stride, p(qsl) if mirrors else None, p(seq), R, T, NB, BS, Hq, Hkv,
                                     D, 0.0, 0, dtype, 0, workspace, ws_bytes, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(qsl=[1, 2], seq=[3]), 2), (dict(qsl=[0, 3, 2], seq=[5, 5]), 2), (dict(qsl=[0, 4], seq=[3]), 2),
    (dict(qsl=[0, 2], seq=[40], stride=2), 2), (dict(qsl=[0, 2], seq=[4], T=3), 2),
    (dict(qsl=[0, 2], seq=[4], D=96), 3), (dict(qsl=[0, 2], seq=[4], Hq=6, Hkv=2), 3),
    (dict(qsl=[0, 2], seq=[4], Hq=5, Hkv=2), 1), (dict(qsl=[0, 2], seq=[4], BS=12), 3),
    (dict(qsl=[0, 2], seq=[4], dtype=7), 1), (dict(qsl=[0, 2], seq=[4], ws_bytes=300), 4),
    (dict(qsl=[0, 2], seq=[4], workspace=None), 4), (dict(qsl=[0, 2], seq=[4], workspace=FAKE + 8), 1),
    (dict(qsl=[0, 2], seq=[4], mirrors=False), 1), (dict(qsl=[0, 2], seq=[4], out=None), 1),
    (dict(qsl=[0, 2], seq=[4], scale_ptr=None), 1), (dict(qsl=[0, 2], seq=[4], scale_ptr=FAKE + 4), 1),
    (dict(qsl=[0, 2], seq=[4], k_new=FAKE), 1),
    (dict(qsl=[0, 200], seq=[300], chunk=0), 4),      # a chunk without scratch for its pages
    (dict(qsl=[0, 200], seq=[300], chunk=100), 4),
    (dict(qsl=[0, 0], seq=[7]), 0), (dict(qsl=[0], seq=[], stride=1), 0),
])
def test_step_refusals(lib, kwargs, status):
    assert step_call(lib, **kwargs) == status
    assert status == 0 or lib.cb_last_error_message()


def test_workspace_size_covers_chunks(lib):
    a = lib.cb_workspace_size_q8(4, 4, 32, 8, 128, 16, 0)
    b = lib.cb_workspace_size_q8(4, 400, 32, 8, 128, 16, 1000)
    assert b - a >= 1000 * 8 * 128 * 4
    assert lib.cb_workspace_size_q8(400, 400, 32, 8, 128, 16, 0) > a


def test_binding_refuses_cpu_and_misshapen_tensors(lib):
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(cb.CbError):
        cb.write_kv_q8(k, k, *(torch.zeros((2, 16, 2, 64), dtype=torch.uint8),) * 2,
                       *(torch.zeros((2, 16, 2), dtype=torch.uint8),) * 2, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(cb.CbError):
        cb.write_kv_q8(k.half(), k, None, None, None, None, None)
