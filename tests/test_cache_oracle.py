"""CPU pins of the cache formats' oracle, and the host checks of the entry points
that write them."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import split_kv_mla_paged_gb300 as mla
from oracle import cache
from split_kv_mla_paged_gb300 import build as mla_build


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load_library()


def test_e4m3_table_and_codes_match_torch():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = cache.e4m3_values()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 9, (20000,), generator=g).float())).clamp(-448, 448)
    assert np.array_equal(cache.e4m3_codes(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_fp4_decode_by_hand():
    page = np.zeros((1, mla.FP4_PAGE_BYTES), np.uint8)
    # Row 3, word 5 (values 40..47, block 1): magnitudes 1..7, 0; values 0, 3 and 6 negative.
    word = sum(m << (4 * j) for j, m in enumerate([1, 2, 3, 4, 5, 6, 7, 0]))
    word |= 1 << 7 | 1 << 31 | 1 << 19
    page[0, 3 * 256 + 20:3 * 256 + 24] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
    page[0, 8192 + 32 * 1 + 3] = 10           # 2^2
    page[0, 8192 + 32 * 2 + 3] = 0x3F         # only the low 4 bits count: NaN
    page[0, 8704 + 64 * 3 + 1] = 0x38         # 1.0
    v = cache.fp4_decode(page)[0, 3]
    assert v[40:48].tolist() == [-2.0, 4.0, 6.0, -8.0, 12.0, 16.0, -24.0, 0.0]
    assert np.isnan(v[64:96]).all() and not np.isnan(v[:64]).any()
    assert v[513] == 1.0


def test_fp4_round_trip_and_half_step():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((64, 576)) * np.exp2(rng.integers(-9, 7, (64, 576 // 32)).repeat(32, 1))
    pool = np.zeros((2, mla.FP4_PAGE_BYTES), np.uint8)
    codes, sc, rope = cache.fp4_encode_rows(x)
    for i in range(64):
        cache.fp4_put(pool, i // 32, i % 32, (codes[i], sc[i], rope[i]))
    v = cache.fp4_decode(pool).reshape(64, 576)
    # Every latent value is within half a step (at most one unit of its scale)
    # of its code unless its block is beyond the largest scale.
    step = np.exp2(sc - 8.0).repeat(32, 1)
    fits = np.abs(x[:, :512]).reshape(64, 16, 32).max(-1).repeat(32, 1) <= 7 * 64
    assert (np.abs(v[:, :512] - x[:, :512]) <= step)[fits].all()
    # Encoding what was decoded gives the same values again.
    codes2, sc2, rope2 = cache.fp4_encode_rows(v)
    pool2 = np.zeros_like(pool)
    for i in range(64):
        cache.fp4_put(pool2, i // 32, i % 32, (codes2[i], sc2[i], rope2[i]))
    assert np.array_equal(cache.fp4_decode(pool2), cache.fp4_decode(pool))


def test_fp4_ties_and_borders():
    # One block per scale border: 7 * 2^k keeps the scale, the next value up takes the next one.
    x = np.zeros((2, 576))
    x[0, 0], x[0, 32], x[0, 64] = 7.0, np.nextafter(7.0, 8), -7.0 * 2 ** -8
    x[0, 96:104] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    x[1, 0], x[1, 32], x[1, 64] = 1e9, np.inf, np.nan
    _, sc, _ = cache.fp4_encode_rows(x)
    assert sc[0, :3].tolist() == [8, 9, 0] and sc[0, 3] == 8
    assert sc[1, :3].tolist() == [14, 14, 15]
    pool = np.zeros((1, mla.FP4_PAGE_BYTES), np.uint8)
    codes, sc, rope = cache.fp4_encode_rows(x)
    for i in range(2):
        cache.fp4_put(pool, 0, i, (codes[i], sc[i], rope[i]))
    v = cache.fp4_decode(pool)[0]
    assert v[0, 0] == 6.0 and v[0, 64] == -6.0 * 2 ** -8
    assert v[0, 96:104].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]
    assert v[1, 0] == 384.0 and v[1, 32] == 384.0 and np.isnan(v[1, 64:96]).all()


def test_rotation_against_complex_product():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2, 576))
    ang = rng.uniform(0, 6, (9, 32))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], axis=1)
    pos = np.array([0, 8, 3, 3, 1])
    w = np.exp(1j * ang[pos])[:, None]
    got = cache.rotate(x, cs, pos, False)[..., 512:]
    z = (x[..., 512::2] + 1j * x[..., 513::2]) * w
    assert np.allclose(got[..., 0::2] + 1j * got[..., 1::2], z, atol=1e-12)
    got = cache.rotate(x, cs, pos, True)[..., 512:]
    z = (x[..., 512:544] + 1j * x[..., 544:]) * w
    assert np.allclose(got[..., :32] + 1j * got[..., 32:], z, atol=1e-12)


def test_kv_append_oracle_agrees_with_the_codes():
    rng = np.random.default_rng(4)
    rows = torch.from_numpy(rng.standard_normal((7, 576)).astype(np.float32)).bfloat16()
    pool = np.zeros((1, 32, 576), np.uint8)
    got, st = oracle.kv_append(rows, np.zeros(7, np.int32), np.arange(7, dtype=np.int32), np.zeros((1, 1), np.int32), pool, 0.5)
    assert st == 0
    assert np.array_equal(got[0, :7], cache.e4m3_codes(rows.double().numpy() / 0.5))


# ---------------------------------------------------------------- host checks
def test_structs_match_the_header(tmp_path):
    import os
    import subprocess
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "mla_decode.h"\nint main(void) {\n'
                   '  printf("%zu", sizeof(mla_prologue_args_t));\n'
                   + "".join(f'  printf(" %zu", offsetof(mla_prologue_args_t, {n}));\n' for n, _ in mla.PrologueArgs._fields_)
                   + '  printf(" %d %d %d %d", MLA_FP4_PAGE_BYTES, MLA_CACHE_FP8, MLA_CACHE_BF16, MLA_CACHE_FP4);\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", header, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = [ctypes.sizeof(mla.PrologueArgs)] + [getattr(mla.PrologueArgs, n).offset for n, _ in mla.PrologueArgs._fields_]
    assert got == want + [mla.FP4_PAGE_BYTES, mla.CACHE_FP8, mla.CACHE_BF16, mla.CACHE_FP4]


FAKE = 1 << 20  # aligned, never dereferenced by the host checks


def _args(**kw):
    a = mla.PrologueArgs(n_tokens=4, positions=FAKE, cos_sin=FAKE, rope_rows=8, kv_rows=FAKE, norm_weight=FAKE,
                         norm_eps=1e-6, max_pages_per_req=2, req_idx=FAKE, page_table=FAKE, kv_pages=FAKE, num_pages=4,
                         batch=1, cache_kind=mla.CACHE_FP8, kv_scale=1.0, q_scale=1.0, q_rows=FAKE, q_out=FAKE,
                         num_heads=12, q_kind=mla.CACHE_FP8)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


@pytest.mark.parametrize("change, word", [
    (dict(n_tokens=-1), "n_tokens"), (dict(kv_rows=None, q_rows=None), "neither"), (dict(rope_halves=2), "rope_halves"),
    (dict(rope_rows=0), "rope_rows"), (dict(cos_sin=None), "rope_rows"), (dict(cos_sin=FAKE + 4), "alignment"),
    (dict(positions=None), "positions"), (dict(kv_row_stride=570), "kv_row_stride"), (dict(kv_row_stride=580), "kv_row_stride"),
    (dict(req_idx=None), "null"), (dict(page_table=None), "null"), (dict(kv_pages=None), "null"), (dict(batch=0), "batch"),
    (dict(max_pages_per_req=0), "batch"), (dict(num_pages=0), "batch"), (dict(kv_rows=FAKE + 2), "alignment"),
    (dict(kv_pages=FAKE + 8), "alignment"), (dict(norm_weight=FAKE + 4), "alignment"), (dict(norm_eps=-1.0), "norm_eps"),
    (dict(norm_eps=float("nan")), "norm_eps"), (dict(cache_kind=3), "cache_kind"),
    (dict(cache_kind=mla.CACHE_BF16, kv_scale=0.5), "kv_scale 1"), (dict(kv_scale=0.0), "normal"),
    (dict(kv_scale=float("inf")), "normal"), (dict(kv_scale=1e-40), "normal"), (dict(kv_scale=2.0 ** 127), "normal"),
    (dict(num_heads=0), "num_heads"), (dict(q_head_stride=-576), "strides"), (dict(q_token_stride=577), "strides"),
    (dict(q_out=None), "q_out"), (dict(q_rows=FAKE + 8), "alignment"), (dict(q_out=FAKE + 8), "alignment"),
    (dict(q_kind=7), "q_kind"), (dict(q_kind=mla.CACHE_BF16, q_scale=2.0), "q_scale 1"), (dict(q_scale=0.0), "normal"),
])
def test_prologue_refusals(lib, change, word):
    assert lib.mla_prologue(_args(**change), None) == mla.MLA_ERR_INVALID_ARG
    assert word in mla.mla_last_error()


def test_prologue_other_refusals(lib):
    assert lib.mla_prologue(None, None) == mla.MLA_ERR_INVALID_ARG
    assert lib.mla_prologue(_args(q_kind=mla.CACHE_FP4), None) == mla.MLA_ERR_UNSUPPORTED
    assert lib.mla_prologue(_args(n_tokens=1 << 40), None) == mla.MLA_ERR_UNSUPPORTED
    assert lib.mla_prologue(_args(n_tokens=0, positions=None), None) == mla.MLA_OK  # touches nothing
    # An empty batch's tensors have null addresses.
    assert lib.mla_prologue(_args(n_tokens=0, positions=None, kv_rows=None, q_rows=None, q_out=None), None) == mla.MLA_OK


def test_decode_fp4_refusals(lib):
    args = [FAKE, FAKE, 4, FAKE, 4, FAKE, FAKE, FAKE, 2, 2, 1, 1, 12, 0, 1.0, 1.0, 0.1, FAKE, 1 << 30, FAKE, None, None]

    def call(opts=None, **at):
        a = list(args)
        for k, v in at.items():
            a[int(k[1:])] = v
        return lib.mla_decode_fp4(*a, None if opts is None else ctypes.byref(opts), None)
    for at in (dict(a0=None), dict(a1=None), dict(a1=FAKE + 8), dict(a2=0), dict(a3=None), dict(a10=0), dict(a8=0), dict(a9=3),
               dict(a16=float("nan")), dict(a17=None), dict(a19=None)):
        assert call(**at) == mla.MLA_ERR_INVALID_ARG, at
    assert call(a11=8, a12=256) == mla.MLA_ERR_UNSUPPORTED  # rows
    assert call(a2=1 << 27) == mla.MLA_ERR_UNSUPPORTED      # pool too large for 32-bit rows
    assert call(a18=16) == mla.MLA_ERR_WORKSPACE_TOO_SMALL
    O = mla.DecodeOptions
    assert call(O(None, None, None, 1.0, None, None, None, FAKE, 2, 1)) == mla.MLA_ERR_UNSUPPORTED
    assert "persistent" in mla.mla_last_error()
    assert call(O(None, None, None, float("inf"))) == mla.MLA_ERR_INVALID_ARG
    assert call(O(None, None, None, 1.0, None, None, None, FAKE, 0)) == mla.MLA_ERR_INVALID_ARG
    assert call(O(None, None, None, 1.0, None, None, None, None, 0, 0, 3)) == mla.MLA_ERR_INVALID_ARG
    # At most batch * max_splits * row groups items.
    assert call(O(None, None, None, 1.0, None, None, None, FAKE, 5), a11=8) == mla.MLA_ERR_INVALID_ARG
    sp = args[:6] + [FAKE, 8] + args[6:]
    assert lib.mla_decode_fp4_sparse(*sp[:6], None, *sp[7:], None, None) == mla.MLA_ERR_INVALID_ARG
    assert lib.mla_decode_fp4_sparse(*sp[:7], 0, *sp[8:], None, None) == mla.MLA_ERR_INVALID_ARG
    assert lib.mla_decode_fp4_sparse(*sp[:20], 16, *sp[21:], None, None) == mla.MLA_ERR_WORKSPACE_TOO_SMALL


def test_pages_copy_refusals(lib):
    def copy(src=FAKE, sp=4, sk=0, dst=2 * FAKE, dp=4, dk=0, si=FAKE, di=FAKE, n=2):
        return lib.mla_pages_copy(src, sp, sk, dst, dp, dk, si, di, None, n, None, None)
    assert copy(n=0, src=None, si=None) == mla.MLA_OK
    for kw in (dict(n=-1), dict(sp=0), dict(dp=0), dict(sk=3), dict(dk=-1), dict(src=None), dict(dst=None), dict(si=None),
               dict(di=None), dict(src=FAKE + 8), dict(dst=FAKE + 8), dict(dk=2, dst=FAKE)):
        assert copy(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    for kw in (dict(sk=1), dict(dk=1), dict(sk=1, dk=2), dict(sk=2, dk=1)):
        assert copy(**kw) == mla.MLA_ERR_UNSUPPORTED, kw
    assert copy(n=1 << 31) == mla.MLA_ERR_UNSUPPORTED


def test_pages_remap_refusals(lib):
    assert lib.mla_pages_remap(None, 0, None, 4, None, None) == mla.MLA_OK
    assert lib.mla_pages_remap(None, 3, FAKE, 4, None, None) == mla.MLA_ERR_INVALID_ARG
    assert lib.mla_pages_remap(FAKE, 3, None, 4, None, None) == mla.MLA_ERR_INVALID_ARG
    assert lib.mla_pages_remap(FAKE, -1, FAKE, 4, None, None) == mla.MLA_ERR_INVALID_ARG
    assert lib.mla_pages_remap(FAKE, 3, FAKE, 0, None, None) == mla.MLA_ERR_INVALID_ARG
    assert lib.mla_pages_remap(FAKE, 1 << 40, FAKE, 4, None, None) == mla.MLA_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_prologue(4, kv_rows=t)
    with pytest.raises(ValueError, match="kv_rows, q_rows"):
        mla.mla_prologue(4)


def test_copy_pages_refuses_clashing_lists():
    pool = torch.zeros(8, 32, 576, dtype=torch.uint8)
    other = torch.zeros(8, mla.FP4_PAGE_BYTES, dtype=torch.uint8)
    with pytest.raises(ValueError, match="two copies"):
        mla.copy_pages(pool, other, [0, 1], [2, 2])
    with pytest.raises(ValueError, match="both a source"):
        mla.copy_pages(pool, pool, [0, 1], [1, 2])
    with pytest.raises(ValueError, match="outside"):
        mla.copy_pages(pool, other, [0, 8], [1, 2])
    with pytest.raises(ValueError, match="outside"):
        mla.copy_pages(pool, other, [0, 1], [1, -1])
    with pytest.raises(ValueError, match="same length"):
        mla.copy_pages(pool, other, [0], [1, 2])
    with pytest.raises(ValueError, match="0..32"):
        mla.copy_pages(pool, other, [0], [1], rows=33)
    with pytest.raises(ValueError, match="32 bits"):
        mla.copy_pages(pool, other, [1 << 32], [1])
    with pytest.raises(ValueError, match="integers"):
        mla.copy_pages(pool, other, [0], [1], rows=2.5)
    mla.copy_pages(pool, other, [], [])
