"""The paged-cache calls on the host: what they refuse before any device work, and the
oracle's quantised rows against values worked out by hand."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import io_aware_exact_07_gb300 as fa
import oracle
from _paged import Batch, check_attn

A = 1 << 20  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    from io_aware_exact_07_gb300 import build
    build.build()
    return fa.load()


CACHE = dict(type=0, num_pages=4, page_size=16, H_kv=2, d=64, sp=2048, sh=1024, sr=64, table=A,
             ts=3, max_pages=3, kv=A)


def common(kw):
    c = dict(CACHE, **{k: v for k, v in kw.items() if k in CACHE})
    return [c[k] for k in CACHE]


def write(lib, k_new=A, v_new=A, k=A, v=A, ks=None, vs=None, cu=A, B=2, T=5, max_q=3, kst=128,
          vst=128, **kw):
    return lib.fa_paged_write(k_new, v_new, k, v, ks, vs, *common(kw), cu, B, T, max_q, kst, vst,
                              None)


def read(lib, k=A, v=A, ks=None, vs=None, B=2, N=20, ko=A, vo=A, **kw):
    return lib.fa_paged_read(k, v, ks, vs, *common(kw), B, N, ko, vo, None)


def attn(lib, q=A, k=A, v=A, ks=None, vs=None, o=A, lse=A, H=4, cu=A, B=2, T=5, max_q=3, qs=256,
         scale=0.125, causal=1, wl=-1, ws=A, wsb=1 << 40, **kw):
    c = common(kw)
    return lib.fa_paged_attn(q, k, v, ks, vs, o, lse, *c[:3], H, *c[3:], cu, B, T, max_q, qs,
                             scale, causal, wl, ws, wsb, None)


@pytest.mark.parametrize("call", [write, read, attn])
@pytest.mark.parametrize("bad,status", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(k=A + 8), 1), (dict(table=0), 1), (dict(kv=0), 1),
    (dict(table=A + 2), 1), (dict(kv=A + 1), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1),
    (dict(page_size=24), 2), (dict(H_kv=0), 1), (dict(d=96), 2), (dict(d=0), 2), (dict(type=2), 2),
    (dict(type=-1), 2), (dict(type=1), 1),  # e4m3 without scales
    (dict(type=1, ks=A), 1), (dict(type=1, ks=A + 8, vs=A), 1), (dict(sp=0), 1), (dict(sh=-64), 1), (dict(sr=60), 1),
    (dict(sp=1 << 40), 1), (dict(type=1, ks=A, vs=A, sr=72), 1),  # 72 codes: not 16-byte rows
    (dict(max_pages=0), 1), (dict(ts=2), 1), (dict(B=0), 1),
    (dict(max_pages=1 << 27, ts=1 << 27), 1),  # positions beyond 32 bits
])
def test_cache_arguments_are_refused(lib, call, bad, status):
    assert call(lib, **bad) == status


def test_new_rows_are_refused(lib):
    for bad in (dict(k_new=0), dict(v_new=A + 4), dict(kst=120), dict(vst=132), dict(T=-1),
                dict(cu=None, T=7), dict(cu=A + 2), dict(max_q=-1)):
        assert write(lib, **bad) == fa.FA_ERR_INVALID_ARG, bad
    assert write(lib, T=0) == fa.FA_OK  # nothing to do, no device needed


def test_read_arguments_are_refused(lib):
    for bad in (dict(N=0), dict(ko=0), dict(vo=A + 8)):
        assert read(lib, **bad) == fa.FA_ERR_INVALID_ARG, bad


def test_attention_arguments_are_refused(lib):
    for bad in (dict(q=0), dict(q=A + 8), dict(o=0), dict(lse=0), dict(lse=A + 2), dict(H=3),
                dict(H=0), dict(qs=248), dict(qs=260), dict(scale=0.0), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(wl=-2), dict(max_q=0), dict(T=-1),
                dict(cu=None, T=5), dict(T=1 << 30)):
        assert attn(lib, **bad) == fa.FA_ERR_INVALID_ARG, bad
    assert attn(lib, H=2 * 129, qs=2 * 129 * 64) == fa.FA_ERR_UNSUPPORTED
    assert attn(lib, T=0) == fa.FA_OK


def test_binding_checks_shapes_types_and_devices():
    # on the CPU every tensor is on the wrong device; the checks before that one still run
    b = Batch([1, 2], [20, 5], 16, 2, 64).on("cpu")
    calls = (lambda **k: fa.paged_write(b.k_new, b.v_new, **k),
             lambda **k: fa.paged_read(N=8, **k), lambda **k: fa.paged_attn(b.q, **k))
    good = dict(k_pages=b.k, v_pages=b.v, page_table=b.table, kv_lens=b.kv)
    for call in calls:
        for bad in (dict(k_pages=b.k[0]), dict(v_pages=b.v[:1]), dict(v_pages=b.v.float()),
                    dict(v_pages=b.v.transpose(1, 2).contiguous().transpose(1, 2)), {}):
            with pytest.raises(ValueError):
                call(**dict(good, **bad))


def test_scale_is_the_smallest_power_of_two_that_holds_the_row():
    x = np.zeros((9, 64))
    x[1, 3], x[2, 3], x[3, 0], x[4, 0] = 448.0, 450.0, 1.75, -1.7578125
    x[5, 0], x[6, 0], x[7, 1], x[8, 5] = 1e30, 2.0 ** -130, np.inf, np.nan
    codes, s = oracle.quantize_rows(x)
    # 448 = 1.75 * 2^8 needs E = 0, 450 E = 1; 1.75 = 448 * 2^-8 needs -8, more than it -7
    assert list(s) == [127, 127, 128, 119, 120, 134, 10, 255, 255]
    assert codes[1, 3] == 0x7E and codes[3, 0] == 0x7E and codes[5, 0] == 0x7E
    assert codes[4, 0] == 0x80 | 0x76  # 1.7578125 * 2^7 = 225: 224 = 1.75 * 2^7, the nearest
    assert np.all(codes[7] == 0x7F) and np.all(codes[0] == 0) and codes[6, 0] == 0
    y = oracle.dequantize_rows(codes, s)
    assert y[2, 3] == 448.0 and y[5, 0] == 57344.0 and np.isnan(y[7:]).all()


def test_dequantised_values_are_exact_in_bf16():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    for byte in (10, 60, 127, 134):
        y = oracle.dequantize_rows(codes[None], np.array([byte], dtype=np.uint8))
        assert np.array_equal(torch.from_numpy(y).to(torch.bfloat16).double().numpy(), y)


def test_paged_oracle_equals_decode_oracle():
    b = Batch([2, 2, 2], [5, 2, 1], 16, 2, 64, G=2, seed=4)
    o, lse, _ = b.oracle(True, 2)
    for i, L in enumerate(b.kv):
        k, v = (np.moveaxis(b.stored(n, i), 0, 1)[None] for n in "kv")
        q = np.moveaxis(b.q[2 * i:2 * i + 2].double().numpy(), 0, 1)[None]
        ro, rl = oracle.fwd_decode(q, k, v, 0.125, causal=True, window_left=2)
        assert np.allclose(np.moveaxis(ro[0], 1, 0), o[2 * i:2 * i + 2], atol=1e-12)
        r = np.moveaxis(rl[0], 1, 0)
        assert np.array_equal(np.isneginf(r), np.isneginf(lse[2 * i:2 * i + 2]))
        assert np.allclose(r[~np.isneginf(r)], lse[2 * i:2 * i + 2][~np.isneginf(r)], atol=1e-12)


def test_attention_check_sees_a_wrong_key():
    # the tolerance of the GPU tests is far below what one key too many or too few changes
    b = Batch([3], [40], 16, 1, 64, seed=6)
    ref = b.oracle(True)
    off = b.oracle(False)
    with pytest.raises(AssertionError):
        check_attn(torch.from_numpy(off[0]), torch.from_numpy(off[1]), ref)
    check_attn(torch.from_numpy(ref[0]).to(torch.bfloat16), torch.from_numpy(ref[1]).float(), ref)


def test_positions_stay_within_32_bits(lib):
    # tables with room for 2^31 - 272 positions, and new tokens that would reach back past -2^31
    room = dict(max_pages=(1 << 27) - 17, ts=1 << 27)
    assert attn(lib, **room, max_q=16) == 1
    assert attn(lib, **room, max_q=15, wsb=0) != 1  # refused for its workspace, or no device


@pytest.mark.parametrize("rows", [[], [[]]])
def test_empty_batches_are_refused(rows):
    kp = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.paged_read(kp, kp, torch.zeros(len(rows), 0, dtype=torch.int32),
                      torch.zeros(len(rows), dtype=torch.int32), 5)


class Captured:
    """Stands for the library: a call gives back its arguments."""
    def __getattr__(self, name):
        return lambda *args: args


@pytest.mark.parametrize("call,name,fmt", [(write, "write", "=24q"), (read, "read", "=20q"),
                                           (attn, "attn", "=25qd4q")])
def test_calls_from_blocks_check_as_the_others_do(lib, call, name, fmt):
    block = getattr(lib, f"fa_paged_{name}_block")
    pack = lambda **kw: struct.pack(fmt, *(0 if v is None else v
                                           for v in call(Captured(), **kw)[:-1]))
    for bad in (dict(k=0), dict(k=A + 8), dict(table=A + 2), dict(kv=0), dict(page_size=24),
                dict(d=96), dict(type=2), dict(type=1), dict(sp=1 << 40), dict(sh=-64),
                dict(max_pages=0), dict(ts=2), dict(B=0), dict(k=A, H_kv=0)):
        assert block(pack(**bad), None) == call(lib, **bad) != 0, bad
    for wide in (dict(B=2 + (1 << 32)), dict(d=64 + (1 << 32)), dict(max_pages=1 << 31)):
        assert block(pack(**wide), None) == 1
    assert block(None, None) == 1


def test_attention_from_a_block_checks_its_own_arguments(lib):
    pack = lambda **kw: struct.pack("=25qd4q", *(0 if v is None else v
                                                 for v in attn(Captured(), **kw)[:-1]))
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=1e300), dict(wl=-2),
                dict(H=3), dict(qs=8), dict(max_q=0), dict(q=A + 2), dict(o=0), dict(wsb=-1)):
        assert lib.fa_paged_attn_block(pack(**bad), None) == 1, bad
