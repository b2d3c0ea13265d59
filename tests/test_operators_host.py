"""Host side of the norm + rotation, the quantised cache, the decode over it
and the selection by length: frequencies, refusals, and the plain
implementations that the GPU tests compare with, pinned against library
routines and differences.  No device is touched."""
import ctypes
import math

import numpy as np
import pytest
import torch

import plain_operators as plain


@pytest.fixture(scope="module")
def bsa():
    import top_block_sparse_bsa_b200 as m
    return m


INVALID, UNSUPPORTED = 1, 2
P = ctypes.c_void_p(4096)       # aligned stand-in; nothing is dereferenced before the checks refuse
ODD = ctypes.c_void_p(4104)


# ------------------------------------------------------------------ frequencies

def test_plain_frequencies(bsa):
    f, s = bsa.bsa_rope_inv_freq(64, 10000.0)
    assert s == 1.0 and f.dtype == torch.float64
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert np.allclose(f.numpy(), want, rtol=1e-14)


def test_scaled_frequencies(bsa):
    base, _ = bsa.bsa_rope_inv_freq(128, 500000.0)
    linear, s = bsa.bsa_rope_inv_freq(128, 500000.0, bsa.BSA_ROPE_LINEAR, 4.0)
    assert s == 1.0 and np.allclose(linear.numpy(), base.numpy() / 4, rtol=1e-14)
    wide, s = bsa.bsa_rope_inv_freq(128, 500000.0, bsa.BSA_ROPE_BASE, 4.0)
    assert s == 1.0 and wide[0] == base[0]
    assert wide[-1].item() == pytest.approx(base[-1].item() / 4, rel=1e-12)
    parts, s = bsa.bsa_rope_inv_freq(128, 500000.0, bsa.BSA_ROPE_PARTS, 8.0, 8192, 32.0, 1.0)
    assert s == pytest.approx(0.1 * math.log(8) + 1, rel=1e-6)
    turns = 8192 * base.numpy() / (2 * math.pi)
    assert np.array_equal(parts.numpy()[turns >= 32], base.numpy()[turns >= 32])
    assert np.allclose(parts.numpy()[turns <= 1], base.numpy()[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(parts.numpy()[mid] < base.numpy()[mid])
    assert np.all(parts.numpy()[mid] > base.numpy()[mid] / 8)
    assert np.all(np.diff(parts.numpy()) < 0)


@pytest.mark.parametrize("args", [(0,), (3,), (64, 0.0), (64, math.inf), (64, 1e4, 4), (64, 1e4, -1),
                                  (64, 1e4, 1, 0.5), (64, 1e4, 1, math.nan), (64, 1e4, 3, 4.0, 0.0),
                                  (64, 1e4, 3, 4.0, 8192, 1.0, 1.0), (64, 1e4, 3, 4.0, 8192, 32.0, 0.0)])
def test_frequency_refusals(bsa, args):
    with pytest.raises(bsa.BsaError) as e:
        bsa.bsa_rope_inv_freq(*args)
    assert e.value.code == INVALID


# --------------------------------------------------------------------- refusals

def _shape(bsa, **kw):
    a = dict(B=2, Hq=8, Hkv=2, Nq=1, Nk=256, d=128, block=64, dtype=bsa.BSA_BF16)
    a.update(kw)
    return bsa.make_shape(a["B"], a["Hq"], a["Hkv"], a["Nq"], a["Nk"], a["d"], a["block"], a["dtype"])


def _encode(bsa, shape, qkv=P, stride=12 * 128, qw=P, kw=P, eps=1e-6, layout=1, rot=128, freq=4096, q=P, k=P, v=P):
    rope = bsa.BsaRope(layout, rot, freq, 1.0)
    return bsa.lib.bsa_qkv_norm_rope(ctypes.byref(shape), qkv, stride, qw, kw, eps, ctypes.byref(rope), None, q, k, v,
                                     None)


def test_encode_refusals(bsa):
    ok = _shape(bsa, Nq=4)
    for kw in (dict(qkv=None), dict(qkv=ODD), dict(stride=12 * 128 - 8), dict(stride=12 * 128 + 4), dict(qw=None),
               dict(kw=None), dict(kw=ODD), dict(eps=-1.0), dict(eps=math.nan), dict(layout=3), dict(layout=-1),
               dict(freq=None), dict(freq=4100), dict(rot=0), dict(rot=136), dict(q=None), dict(k=ODD),
               dict(v=None)):
        assert _encode(bsa, ok, **kw) == INVALID, kw
    for kw in (dict(rot=12), dict(rot=4)):
        assert _encode(bsa, ok, **kw) == UNSUPPORTED, kw
    assert _encode(bsa, _shape(bsa, Nq=0)) == INVALID
    assert _encode(bsa, _shape(bsa, Nq=4, dtype=7)) == INVALID
    assert _encode(bsa, _shape(bsa, Nq=4, d=100), rot=96) == UNSUPPORTED
    assert _encode(bsa, _shape(bsa, Nq=4, d=264), stride=12 * 264) == UNSUPPORTED
    assert _encode(bsa, _shape(bsa, B=1 << 16, Nq=1 << 16)) == UNSUPPORTED
    assert bsa.lib.bsa_qkv_norm_rope(None, P, 1536, None, None, 0.0, None, None, P, P, P, None) == INVALID


def test_encode_backward_refusals(bsa):
    ok = _shape(bsa, Nq=4)
    rope = bsa.BsaRope(1, 128, 4096, 1.0)

    def call(dq=P, dv=P, d_qkv=P, stride=12 * 128, qw=P, kw=P, dqw=P, dkw=P, ws=P, size=1 << 30):
        return bsa.lib.bsa_qkv_norm_rope_bwd(ctypes.byref(ok), P, 12 * 128, qw, kw, 1e-6, ctypes.byref(rope), None, dq,
                                             P, dv, d_qkv, stride, dqw, dkw, ws, size, None)
    for kw in (dict(dq=None), dict(dv=ODD), dict(d_qkv=None), dict(d_qkv=ODD), dict(stride=128), dict(dqw=None),
               dict(dkw=None), dict(ws=None), dict(ws=ODD), dict(qw=None, kw=None)):
        assert call(**kw) == INVALID, kw


def test_quant_cache_refusals(bsa):
    def append(shape, k=P, v=P, lens=P, table=P, stride=4, pages=8, kp=P, vp=ctypes.c_void_p(8192), ke=P,
               ve=ctypes.c_void_p(8192), pooled=None):
        return bsa.lib.bsa_paged_append_quant(ctypes.byref(shape), k, v, lens, None, table, stride, pages, kp, vp, ke,
                                              ve, pooled, None)
    ok = _shape(bsa)
    for kw in (dict(k=None), dict(v=ODD), dict(lens=None), dict(table=None), dict(stride=0), dict(pages=0),
               dict(kp=None), dict(kp=ODD), dict(vp=P), dict(ve=P), dict(ke=None), dict(ve=ODD), dict(pooled=ODD)):
        assert append(ok, **kw) == INVALID, kw
    for kw in (dict(dtype=bsa.BSA_F32), dict(d=100), dict(d=264), dict(block=128)):
        assert append(_shape(bsa, **kw)) == UNSUPPORTED, kw
    assert append(ok, pages=1 << 28) == UNSUPPORTED

    def read(shape, lens=P, ko=P, vo=P, pages=8):
        return bsa.lib.bsa_paged_read_quant(ctypes.byref(shape), P, P, P, P, pages, P, 4, lens, None, ko, vo, None)
    for kw in (dict(lens=None), dict(ko=None, vo=None), dict(ko=ODD), dict(vo=ODD), dict(pages=0)):
        assert read(ok, **kw) == INVALID, kw
    assert read(_shape(bsa, block=32)) == UNSUPPORTED


def test_quant_decode_refusals(bsa):
    def call(shape, q=P, stride=4, idx=P, idx_stride=3, scale=0.1, ws=P, size=1 << 30, o=P, pages=8):
        return bsa.lib.bsa_sparse_attn_decode_quant(ctypes.byref(shape), q, P, P, P, P, pages, P, stride, None, idx,
                                                    idx_stride, scale, ws, size, o, None, None)
    ok = _shape(bsa)
    for kw in (dict(q=None), dict(q=ODD), dict(o=None), dict(stride=3), dict(idx_stride=0), dict(idx=None),
               dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf), dict(ws=None), dict(ws=ODD)):
        assert call(ok, **kw) == INVALID, kw
    assert call(_shape(bsa, Nq=2)) == INVALID
    for kw in (dict(dtype=bsa.BSA_F32), dict(d=96), dict(Hq=34), dict(B=8193), dict(block=128)):
        assert call(_shape(bsa, **kw), stride=100000) == UNSUPPORTED, kw
    assert call(ok, pages=1 << 28) == UNSUPPORTED


def test_select_by_length_refusals(bsa):
    def call(scores=P, rows=8, ncols=4, lens=P, per=2, block=64, kb=2, idx=P, stride=3):
        return bsa.lib.bsa_topk_select_lens(scores, rows, ncols, lens, per, block, kb, idx, stride, None, None)
    for kw in (dict(scores=None), dict(rows=-1), dict(ncols=0), dict(lens=None), dict(per=0), dict(per=3),
               dict(block=0), dict(kb=-1), dict(idx=None), dict(stride=2)):
        assert call(**kw) == INVALID, kw
    assert call(ncols=8193) == UNSUPPORTED
    assert call(rows=0) == 0


# -------------------------------------------- the plain implementations themselves

def _encode_case(layout, weights=True, B=2, N=3, Hq=4, Hkv=2, d=16, rot=8, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    qkv = r(B, N, Hq + 2 * Hkv, d)
    w = (1 + 0.2 * r(d), 1 + 0.2 * r(d)) if weights else (None, None)
    pos = torch.randint(-50, 100000, (B, N), generator=g)
    freq = 100.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    grads = r(B, Hq, N, d), r(B, Hkv, N, d), r(B, Hkv, N, d)
    return (qkv, Hq, Hkv, *w, 1e-5, freq, layout, pos, 1.3), grads


@pytest.mark.parametrize("layout", ["none", "half", "pairs"])
@pytest.mark.parametrize("weights", [True, False])
def test_plain_encode_gradient_is_autograd_and_differences(layout, weights):
    args, grads = _encode_case(layout, weights)
    got, _ = plain.encode_grad(*args, *grads)
    leaves = [args[0].clone().requires_grad_()] + [w.clone().requires_grad_() for w in args[3:5] if w is not None]
    full = (leaves[0], *args[1:3], *(leaves[1:] if weights else (None, None)), *args[5:])
    torch.autograd.backward(plain.encode(*full), grads)
    for x, w in zip(leaves, got):
        assert torch.allclose(x.grad, w, rtol=1e-10, atol=1e-12)

    def loss(a):
        return sum((o * g).sum() for o, g in zip(plain.encode(*a), grads))
    step = 1e-6
    for n, place in ((0, (1, 2, 1, 3)), (0, (0, 1, 5, 9)), (0, (0, 0, 7, 2))) + (((3, (5,)), (4, (0,))) if weights else ()):
        sides = []
        for sign in (1, -1):
            a = list(args)
            a[n] = a[n].clone()
            a[n][place] += sign * step
            sides.append(loss(a))
        slope = (sides[0] - sides[1]) / (2 * step)
        want = got[0 if n == 0 else n - 2][place]
        assert abs(slope - want) <= 1e-6 * (1 + abs(want))


def test_plain_rotation_keeps_products_by_distance():
    # rotated rows' products depend on the positions' difference alone, and a turned pair keeps its length
    args, _ = _encode_case("half", False, B=1, N=2, Hq=1, Hkv=1, rot=16)
    dots = []
    for shift in (0, 1234):
        a = list(args)
        a[8] = torch.tensor([[7 + shift, 3 + shift]])
        a[9] = 1.0
        q, k, _ = plain.encode(*a)
        dots.append((q[0, 0, 0] @ k[0, 0, 1]).item())
        assert torch.allclose(q.norm(dim=-1), a[0][:, :, 0].norm(dim=-1)[:, None])
    assert dots[0] == pytest.approx(dots[1], abs=1e-9)


def test_plain_codes_are_the_library_s_float8():
    x = torch.from_numpy(plain.E4M3.copy()).float()
    assert torch.equal(torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().isnan(), x.isnan())
    lib = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    assert torch.equal(lib[~x.isnan()], x[~x.isnan()])
    g = torch.Generator().manual_seed(1)
    rows = (torch.randn((200, 64), generator=g) * torch.exp(4 * torch.randn((200, 1), generator=g))).bfloat16()
    codes, exps = plain.quantise(rows.double().numpy())
    y = rows.float() / 2.0 ** (torch.from_numpy(exps).float() - 127)[:, None]
    assert y.abs().max() <= 448 and np.all(np.abs(y.numpy()).max(1) > 224)
    assert np.array_equal(y.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), codes)


def test_plain_quantise_corners():
    codes, exps = plain.quantise(np.array([[0.0, -0.0], [448.0, 1.0], [449.0, 1.0], [np.inf, 2.0], [np.nan, -2.0]]))
    assert exps.tolist() == [10, 127, 128, 120, 120]
    assert codes[0].tolist() == [0, 128] and codes[1, 0] == 126
    assert codes[3, 0] == 127 and codes[4, 0] == 127
    assert plain.dequantise(codes, exps)[3, 1] == 2.0 and plain.dequantise(codes, exps)[4, 1] == -2.0


def test_plain_decode_is_the_library_s_attention():
    r = np.random.default_rng(0)
    codes = r.integers(0, 126, (9, 2, 64, 64), dtype=np.uint8) | (r.integers(0, 2, (9, 2, 64, 64), dtype=np.uint8) << 7)
    exps = r.integers(117, 121, (9, 2, 64), dtype=np.uint8)
    table, lens = np.array([[3, 1, 8], [0, 7, 2]]), [130, 64]
    q = r.standard_normal((2, 4, 64))
    o, lse, _, _ = plain.decode(q, codes, codes, exps, exps, table, lens, None, 0.1)
    for b in range(2):
        kv = torch.from_numpy(plain.dequantise(codes[table[b]], exps[table[b]])).transpose(0, 1).reshape(2, -1, 64)
        kv = kv[:, :lens[b]].repeat_interleave(2, 0)
        want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[b])[:, None], kv, kv, scale=0.1)
        assert np.allclose(o[b], want[:, 0].numpy(), rtol=1e-9)
        assert np.allclose(lse[b], torch.logsumexp(torch.einsum("hd,hnd->hn", torch.from_numpy(q[b]), kv) * 0.1, -1))


def test_plain_select_is_the_oracle_s_on_whole_blocks():
    import oracle
    r = np.random.default_rng(3)
    s = r.integers(-3, 4, (6, 20)).astype(np.float32)
    s[0, ::3] = np.nan
    want, cnt = oracle.topk(s, 1, 5, idx_stride=7)
    got, n = plain.select(s, [20 * 64] * 3, 2, 64, 5, 7)
    assert np.array_equal(got, want) and np.array_equal(n, cnt)


# ------------------------------------------------------------------ step objects

def test_steps_refuse_shapes_that_do_not_match(bsa):
    from top_block_sparse_bsa_b200 import pipeline
    qkv = torch.zeros((2, 3, 8, 64))
    with pytest.raises(ValueError):
        pipeline.QkvStep(qkv, 4, 1)
    with pytest.raises(ValueError):
        pipeline.QkvStep(qkv, 4, 2, positions=torch.zeros((3, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        pipeline.QkvStep(qkv, 4, 2, q_weight=torch.ones(32), k_weight=torch.ones(64))
    step = pipeline.QkvStep(qkv, 4, 2)
    with pytest.raises(ValueError):
        step.backward(torch.zeros((2, 4, 3, 64)), torch.zeros((2, 4, 3, 64)), torch.zeros((2, 2, 3, 64)))
    with pytest.raises(ValueError):
        bsa.make_rope(bsa.BSA_ROPE_HALF)
    with pytest.raises(ValueError):
        bsa.make_rope(bsa.BSA_ROPE_HALF, torch.zeros(8))
    q, pool = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((5, 2, 64, 128), dtype=torch.uint8)
    with pytest.raises(ValueError):
        pipeline.QuantDecodeStep(q, pool, pool, pool[..., 0], pool[..., 0], torch.zeros((2, 2), dtype=torch.int32),
                                 torch.zeros(2, dtype=torch.int32))
