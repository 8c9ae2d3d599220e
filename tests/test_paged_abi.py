"""Host-side checks of the paged-cache calls (nothing is launched, no GPU is needed) and the rotary table."""

import ctypes as C
import os

import numpy as np
import pytest

from indexer_driven_sparse_gb300 import binding as qb
from indexer_driven_sparse_gb300 import build as qbuild
from oracle import paged_oracle as P

FAKE = 0x10000000  # never dereferenced: every call below fails or returns before a launch
BAD, UNSUPPORTED, SMALL = qb.QSA_ERR_INVALID_ARGUMENT, qb.QSA_ERR_UNSUPPORTED, qb.QSA_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qb.load()


def rope_cfg(**kw):
    base = dict(head_dim=128, rot_begin=0, rot_dim=128, interleaved=0, scaling=0, original_len=4096, base=1e4, factor=4.0,
                beta_fast=32.0, beta_slow=1.0)
    base.update(kw)
    return qb.qsa_rope_config(*[base[n] for n, _ in qb.qsa_rope_config._fields_])


def table_of(lib, cfg):
    phase = np.zeros(max(cfg.rot_dim // 2, 1), np.uint64)
    amp = C.c_float(-1)
    st = lib.qsa_rope_table(C.byref(cfg), phase.ctypes.data, C.byref(amp))
    return st, phase[: cfg.rot_dim // 2], amp.value


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "by_parts"])
@pytest.mark.parametrize("rot,base", [(128, 1e4), (64, 1e6), (256, 5e5), (16, 100.0)])
def test_rope_table_against_64_bits(lib, scaling, rot, base):
    cfg = rope_cfg(head_dim=256, rot_dim=rot, base=base, scaling=qb.ROPE_SCALINGS.index(scaling), factor=8.0)
    st, phase, amp = table_of(lib, cfg)
    assert st == qb.QSA_OK
    freq, want_amp = P.rope_frequencies(rot, base, scaling, 8.0, 4096)
    # a frequency carries a few rounding errors of 64-bit arithmetic, and the table's last bit is 2^-64 of a turn
    # (5.4e-20, cut off): for the slowest pairs, of 1e-6 turns a token, that is the larger part
    turns = phase.astype(np.float64) * 2.0 ** -64
    assert np.all(np.abs(turns - freq / (2 * np.pi)) <= 1e-14 * freq + 2.0 ** -64)
    assert abs(amp - want_amp) <= 2.0 ** -24 * want_amp


def test_rope_table_holds_far_positions(lib):
    st, phase, _ = table_of(lib, rope_cfg(base=1e6))
    for p in (3_145_727, 2 ** 31 - 1, -12345):
        angle = (phase * np.uint64(p & (2 ** 64 - 1))).astype(np.float64) * 2.0 ** -64 * 2 * np.pi
        want = p * P.rope_frequencies(128, 1e6)[0]
        # the 64-bit frequency is off by a few 2^-53 of itself, on both sides
        assert np.all(np.abs(np.exp(1j * angle) - np.exp(1j * want)) <= abs(p) * 4e-15 + 1e-12)


@pytest.mark.parametrize("bad,code", [
    (dict(head_dim=120), UNSUPPORTED), (dict(head_dim=2048), UNSUPPORTED), (dict(rot_dim=24), UNSUPPORTED),
    (dict(rot_begin=4, rot_dim=64), UNSUPPORTED), (dict(rot_begin=-8, rot_dim=64), UNSUPPORTED),
    (dict(rot_begin=16), BAD), (dict(base=1.0), BAD), (dict(base=float("nan")), BAD), (dict(scaling=4), BAD),
    (dict(scaling=-1), BAD), (dict(scaling=1, factor=0.0), BAD), (dict(scaling=3, original_len=0), BAD),
    (dict(scaling=3, beta_fast=1.0), BAD), (dict(scaling=3, beta_slow=0.0), BAD)])
def test_rope_table_refusals(lib, bad, code):
    assert table_of(lib, rope_cfg(**bad))[0] == code
    assert b"qsa_rope_table" in lib.qsa_last_error()


def test_rope_refusals(lib):
    cfg = rope_cfg()

    def call(cfg=cfg, phase=FAKE, x=FAKE, x_ld=512, pos=FAKE, n=3, heads=4, out=FAKE + 64, out_ld=512):
        return lib.qsa_rope(C.byref(cfg) if cfg else None, phase, 1.0, x, x_ld, pos, n, heads, out, out_ld, None)

    assert call(n=0) == qb.QSA_OK and call(heads=0) == qb.QSA_OK
    for kw in (dict(cfg=None), dict(n=-1), dict(heads=-1), dict(x=0), dict(x=FAKE + 8), dict(x_ld=504), dict(x_ld=516),
               dict(out=0), dict(out=FAKE + 2), dict(out_ld=256), dict(pos=0), dict(pos=FAKE + 2), dict(phase=0),
               dict(phase=FAKE + 8), dict(out=FAKE, out_ld=520)):
        assert call(**kw) == BAD, kw
    assert call(heads=70000, x_ld=70000 * 128, out_ld=70000 * 128) == UNSUPPORTED


def paged_cfg(**kw):
    base = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, softmax_scale=0.0, window=0)
    base.update(kw)
    return qb.make_paged_config(**base)


GEOMETRY = [(dict(head_dim=96), UNSUPPORTED), (dict(n_q_heads=9), UNSUPPORTED), (dict(n_q_heads=34), UNSUPPORTED),
            (dict(n_q_heads=0), BAD), (dict(n_kv_heads=0), BAD), (dict(page_size=0), BAD), (dict(window=-1), BAD),
            (dict(softmax_scale=float("inf")), BAD), (dict(softmax_scale=float("nan")), BAD),
            (dict(n_q_heads=8192, n_kv_heads=512), UNSUPPORTED)]


def decode(lib, cfg, fp8=False, q=FAKE, q_ld=1024, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=10, table=FAKE, ld=4,
           lens=FAKE, B=3, out=FAKE, ws=FAKE, bytes=1 << 30):
    c = C.byref(cfg) if cfg else None
    if fp8:
        return lib.qsa_paged_decode_fp8kv(c, q, q_ld, k, ks, v, vs, pages, table, ld, lens, B, out, 0, ws, bytes, None)
    return lib.qsa_paged_decode(c, q, q_ld, k, v, pages, table, ld, lens, B, out, 0, ws, bytes, None)


@pytest.mark.parametrize("bad,code", GEOMETRY)
def test_paged_geometry_refused(lib, bad, code):
    cfg = paged_cfg(**bad)
    assert decode(lib, cfg) == code
    assert lib.qsa_paged_workspace_size(C.byref(cfg)) == 0
    assert lib.qsa_paged_workspace_size(None) == 0


def test_paged_decode_refusals(lib):
    cfg = paged_cfg()
    assert decode(lib, cfg, B=0) == qb.QSA_OK
    for kw in (dict(cfg=None), dict(B=-1), dict(B=65536), dict(q=0), dict(q=FAKE + 8), dict(q_ld=1016), dict(q_ld=1028),
               dict(k=0), dict(v=0), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(table=0), dict(lens=0), dict(out=0),
               dict(out=FAKE + 4), dict(pages=-1), dict(ld=-1), dict(ws=0), dict(ws=FAKE + 16), dict(table=FAKE + 2),
               dict(lens=FAKE + 1)):
        assert decode(lib, kw.pop("cfg", cfg), **kw) == BAD, kw
    assert decode(lib, cfg, bytes=255) == SMALL
    assert decode(lib, cfg, pages=1 << 28) == UNSUPPORTED
    assert decode(lib, paged_cfg(head_dim=64), fp8=True, q_ld=512) == UNSUPPORTED
    for kw in (dict(ks=0), dict(vs=0), dict(ks=FAKE + 4), dict(vs=FAKE + 4)):
        assert decode(lib, cfg, fp8=True, **kw) == BAD, kw


def test_rope_append_refusals(lib):
    cfg, rope = paged_cfg(), rope_cfg()

    def call(fp8=False, cfg=cfg, rope=rope, phase=FAKE, q=FAKE, q_ld=1024, k=FAKE, k_ld=256, v=FAKE, v_ld=256, pos=FAKE,
             n=3, q_out=FAKE + 64, q_out_ld=1024, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pages=10, table=FAKE, ld=4, rows=3,
             ws=FAKE, bytes=1 << 30):
        c, r = C.byref(cfg) if cfg else None, C.byref(rope) if rope else None
        head = (c, r, phase, 1.0, q, q_ld, k, k_ld, v, v_ld, 0, pos, n, q_out, q_out_ld)
        tail = (pages, table, ld, rows, ws, bytes, None)
        if fp8:
            return lib.qsa_rope_append_fp8kv(*head, kc, ks, vc, vs, *tail)
        return lib.qsa_rope_append(*head, kc, vc, *tail)

    assert call(n=0) == qb.QSA_OK
    for kw in (dict(cfg=None), dict(rope=None), dict(rope=rope_cfg(head_dim=256)), dict(n=-1), dict(rows=-1),
               dict(q=FAKE + 8), dict(q_ld=8), dict(q_out=0), dict(q_out=FAKE, q_out_ld=1032), dict(k=0), dict(k_ld=248),
               dict(v=0), dict(v=FAKE + 2), dict(v_ld=260), dict(pos=0), dict(table=0), dict(phase=0), dict(phase=FAKE + 8), dict(kc=0),
               dict(vc=0), dict(kc=FAKE + 8), dict(ws=0), dict(ws=FAKE + 128), dict(pages=-1), dict(ld=-1), dict(pos=FAKE + 2), dict(table=FAKE + 1)):
        assert call(**kw) == BAD, kw
    for kw in (dict(ks=0), dict(vs=0), dict(ks=FAKE + 4), dict(kc=FAKE + 8)):
        assert call(fp8=True, **kw) == BAD, kw
    assert call(bytes=16) == SMALL
    assert call(cfg=paged_cfg(head_dim=64), rope=rope_cfg(head_dim=64, rot_dim=64), fp8=True) == UNSUPPORTED


def test_page_calls_refusals(lib):
    def planes(**kw):
        base = dict(base=FAKE, plane_stride=4096, page_bytes=64, n_planes=2)
        base.update(kw)
        return (qb.qsa_page_planes * 1)(qb.qsa_page_planes(**base))

    def fork(ps=4, parent=FAKE, add=FAKE, n_out=3, table=FAKE, lens=FAKE, n_in=3, ld=4, ref=FAKE, pages=9, t_out=FAKE + 256,
             l_out=FAKE + 256, r_out=FAKE + 256, groups=None, n=1, ws=FAKE, bytes=1 << 30):
        return lib.qsa_fork_pages(ps, parent, add, n_out, table, lens, n_in, ld, ref, pages, t_out, l_out, r_out,
                                  planes() if groups is None else groups, n, ws, bytes, None)

    def compact(ps=4, table=FAKE, lens=FAKE, rows=3, ld=4, ref=FAKE, pages=9, t_out=FAKE, r_out=FAKE + 256, groups=None, n=1,
                ws=FAKE, bytes=1 << 30):
        return lib.qsa_compact_pages(ps, table, lens, rows, ld, ref, pages, t_out, r_out,
                                     planes() if groups is None else groups, n, ws, bytes, None)

    bad_groups = [dict(groups=planes(base=0)), dict(groups=planes(page_bytes=6)), dict(groups=planes(base=FAKE + 4)),
                  dict(groups=planes(plane_stride=4100)), dict(groups=planes(n_planes=-1)), dict(n=9), dict(n=-1),
                  dict(groups=planes(page_bytes=-16)), dict(groups=planes(page_bytes=36, base=FAKE + 2))]
    for kw in [dict(ps=0), dict(parent=0), dict(add=0), dict(n_out=-1), dict(n_out=65537), dict(n_in=65537), dict(table=0),
               dict(lens=0), dict(ld=-1), dict(ref=0), dict(pages=-1), dict(t_out=0), dict(t_out=FAKE), dict(l_out=0),
               dict(l_out=FAKE), dict(r_out=0), dict(r_out=FAKE), dict(parent=FAKE + 2), dict(r_out=FAKE + 1), dict(ws=0), dict(ws=FAKE + 64)] + bad_groups:
        assert fork(**kw) == BAD, kw
    for kw in [dict(ps=0), dict(table=0), dict(lens=0), dict(rows=-1), dict(rows=65537), dict(ld=-1), dict(ref=0),
               dict(pages=-1), dict(t_out=0), dict(r_out=0), dict(r_out=FAKE), dict(ws=0)] + bad_groups:
        assert compact(**kw) == BAD, kw
    assert fork(bytes=256) == SMALL and compact(bytes=256) == SMALL
    assert fork(pages=(1 << 30) + 1) == UNSUPPORTED and compact(pages=(1 << 30) + 1) == UNSUPPORTED
    assert fork(n_out=0, n_in=0, pages=0) == qb.QSA_OK and compact(rows=0, pages=0) == qb.QSA_OK
    assert lib.qsa_pages_workspace_size(-1, 5) == 0 and lib.qsa_pages_workspace_size(5, -1) == 0
    assert lib.qsa_pages_workspace_size(65537, 5) == 0

    def copy(src=FAKE, dst=FAKE, n=3, groups=None, to=None, count=1, ws=FAKE, bytes=256):
        return lib.qsa_copy_pages(src, dst, n, planes() if groups is None else groups, 9, to, 9, count, ws, bytes, None)

    assert copy(n=0) == qb.QSA_OK and copy(count=0) == qb.QSA_OK
    for kw in [dict(src=0), dict(dst=0), dict(src=FAKE + 2), dict(n=-1), dict(ws=0), dict(to=planes(n_planes=3)), dict(to=planes(page_bytes=32)),
               dict(count=9)] + [dict(groups=g["groups"]) for g in bad_groups if "groups" in g]:
        assert copy(**kw) == BAD, kw
    assert copy(bytes=100) == SMALL


def test_binding_refuses_wrong_tensors(lib):
    import torch
    bf16 = dict(dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    rope = qb.rope_table(128, device="cpu")
    x, pos = torch.zeros(2, 8, 128, **bf16), torch.zeros(2, **i32)

    def refused(error, text, fn, *args):
        with pytest.raises(error, match=text):
            fn(*args)

    # everything right but the device
    refused(ValueError, "x is on cpu", qb.qsa_rope, rope, x, pos, x)
    refused(TypeError, "x must be torch.BFloat16", qb.qsa_rope, rope, x.float(), pos, x)
    refused(TypeError, "x must be a tensor", qb.qsa_rope, rope, None, pos, x)
    refused(ValueError, "x must be", qb.qsa_rope, rope, x[0], pos, x)
    refused(ValueError, r"x must be \[2, 8, 128\], got \[2, 8, 64\]", qb.qsa_rope, rope, x[..., :64], pos, x)
    refused(ValueError, "heads of x", qb.qsa_rope, rope, torch.zeros(8, 2, 128, **bf16).transpose(0, 1), pos, x)
    refused(ValueError, "heads of x", qb.qsa_rope, rope, torch.zeros(2, 8, 256, **bf16)[..., ::2], pos, x)
    cfg = paged_cfg(n_q_heads=8, n_kv_heads=2)
    kv = [torch.zeros(5, 16, 2, 128, **bf16) for _ in range(2)]
    table, lens, ws = torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(512, dtype=torch.uint8)
    lse = torch.zeros(2, 8)

    def decode(cfg=cfg, q=x, kv=kv, table=table, lens=lens, out=x, lse=lse, ws=ws):
        qb.qsa_paged_decode(cfg, q, *kv, table, lens, out, lse, ws)

    for error, text, kw in ((ValueError, "q is on cpu", {}), (TypeError, "qsa_paged_config", dict(cfg=rope.cfg)),
                            (TypeError, "table must be torch.Int", dict(table=table.long())),
                            (ValueError, "table must have two", dict(table=lens)),
                            (ValueError, r"q must be \[3", dict(table=torch.zeros(3, 3, **i32)))):
        with pytest.raises(error, match=text):
            decode(**kw)
    planes = [torch.zeros(3, 6, 4)]
    ref = torch.zeros(6, **i32)
    refused(ValueError, "parent is on cpu", qb.qsa_fork_pages, 4, pos, pos, table, lens, ref, table, lens, ref, planes, ws)
    refused(ValueError, "table is on cpu", qb.qsa_compact_pages, 4, table, lens, ref, table, ref, planes, ws)
    refused(ValueError, "src is on cpu", qb.qsa_copy_pages, pos, pos, planes, ws)
    with pytest.raises(ValueError):
        qb.rope_table(128, scaling="other")
    with pytest.raises(qb.QsaError):
        qb.rope_table(120, device="cpu")
    t = qb.rope_table(128, 64, device="cpu")
    assert t.phase.shape == (32,) and t.amplitude == 1.0


@pytest.mark.parametrize("rot,base,trained,lo,hi", [
    # by hand: c(b) = rot / 2 x ln(trained / (2 pi b)) / ln(base)
    (128, 1e4, 131072, 45, 70),    # c(32) = 64 x 6.4798 / 9.2103 = 45.03, c(1) = 64 x 9.9456 / 9.2103 = 69.11: past pair 63
    (64, 1e4, 262144, 24, 37),     # c(32) = 32 x 7.1730 / 9.2103 = 24.92, c(1) = 32 x 10.6387 / 9.2103 = 36.96: past pair 31
    (16, 100.0, 65536, 10, 15),    # c(32) = 8 x 5.7867 / 4.6052 = 10.05, c(1) = 8 x 9.2525 / 4.6052 = 16.07: 17, but at most 15
    (128, 1e6, 32768, 23, 40)])    # c(32) = 64 x 5.0936 / 13.8155 = 23.60, c(1) = 64 x 8.5593 / 13.8155 = 39.65: inside
def test_rope_by_parts_ramp_may_end_past_the_last_pair(lib, rot, base, trained, lo, hi):
    """Frequencies of scaling by parts against the ramp's ends worked out by hand."""
    cfg = rope_cfg(head_dim=256, rot_dim=rot, base=base, scaling=qb.ROPE_SCALINGS.index("by_parts"), factor=4.0,
                   original_len=trained)
    st, phase, amp = table_of(lib, cfg)
    assert st == qb.QSA_OK and abs(amp - (0.1 * np.log(4.0) + 1.0)) < 1e-6
    i = np.arange(rot // 2)
    g = np.clip((i - lo) / (hi - lo), 0.0, 1.0)
    want = base ** (-2.0 * i / rot) * (1.0 - 0.75 * g)
    turns = phase.astype(np.float64) * 2.0 ** -64
    assert np.all(np.abs(turns - want / (2 * np.pi)) <= 1e-14 * want + 2.0 ** -64)
    if rot == 128 and base == 1e4:                        # pair 63: g = 18 / 25, 1e4^(-126/128) x 0.46
        assert abs(turns[63] * 2 * np.pi - 5.3119e-5) < 1e-8


def test_kernels_that_begin_early_use_no_read_only_loads():
    """The paged kernels start while the one before them still writes lengths, tables and rows: of all they read only the
    rotary phases may come through the read-only path."""
    for name in ("paged.cuh", "paged_decode.cu", "pages.cu", "rope.cu"):
        with open(os.path.join(qbuild.CSRC, name)) as f:
            code = [line.split("//")[0] for line in f]
        assert not any("ld.global.nc" in line or "ldg_nc" in line for line in code), name
        assert all("r.phase" in line for line in code if "__ldg(" in line), name


@pytest.mark.parametrize("bad", [dict(scaling=1, factor=1e-320), dict(scaling=2, factor=1e-300, rot_dim=16),
                                 dict(scaling=2, factor=1e300, rot_dim=16), dict(scaling=3, factor=5e-324)])
def test_rope_table_refuses_factors_out_of_range(lib, bad):
    """A frequency that is no number has no fraction of a turn."""
    assert table_of(lib, rope_cfg(**bad))[0] == BAD
    assert b"factor" in lib.qsa_last_error()


def test_corrected_quotient_of_bf16_values_is_correctly_rounded():
    """The FP8 append divides x by scale = RN(amax / 448) as q = RN(x RN(1 / scale)), then RN(q + RN(x - q scale) RN(1 / scale))
    with fused multiply-adds: the correctly rounded quotient for all pairs of bf16 significands, and one unit in the last
    place off at most for 24-bit x. fp32 operations round once; the products below have 48 bits and the remainder
    cancels, so both are exact in fp64; the last sum is checked not to lie where rounding it twice could matter."""
    f32, f64 = np.float32, np.float64
    rng = np.random.default_rng(0)
    short = np.arange(128, 256, dtype=f32) / f32(128)
    wide = rng.integers(1 << 23, 1 << 24, 512).astype(f32) / f32(1 << 23)
    for a in short:
        scale = f32(a / f32(448))
        inv = f32(f32(1) / scale)
        for xs in (short, wide):
            q = xs * inv
            rest = (xs.astype(f64) - q.astype(f64) * f64(scale)).astype(f32)
            total = q.astype(f64) + rest.astype(f64) * f64(inv)
            got = total.astype(f32)
            want = xs / scale
            ulp = np.spacing(want)
            assert got.dtype == want.dtype == f32 and q.dtype == f32
            # fp64 rounds `total` by 2^-53 of it, far less than its distance to the middle between two fp32 values
            assert np.all(np.abs(np.abs(total - got.astype(f64)) - ulp / f64(2)) > f64(2) ** -48 * total)
            assert np.array_equal(got, want) if xs is short else np.all(np.abs(got - want) <= ulp)
