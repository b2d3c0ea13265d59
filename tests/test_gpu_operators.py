"""GPU parity of the norm + rotation (and its backward), the quantised paged
cache, the decode over it and the selection by length, against the plain
64-bit implementations; then as they are used together: projection ->
prefill -> both backwards, and a ragged decode loop.

Tolerances count roundings.  Half a step of a type is finfo(t).eps / 2
relative to the value: bf16 2^-8, fp32 2^-24.
"""
import math

import numpy as np
import pytest
import torch

import plain_operators as plain

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def bsa():
    import top_block_sparse_bsa_b200 as m
    return m


@pytest.fixture(scope="module")
def pipe():
    from top_block_sparse_bsa_b200 import pipeline
    return pipeline


@pytest.fixture(autouse=True)
def status_is_clean(bsa):
    yield
    code, flags = bsa.bsa_device_status(reset=True)
    assert code == 0 and flags == 0, f"device status {code} flags {flags:#x}"


def _flagged(bsa):
    code, flags = bsa.bsa_device_status(reset=True)
    assert code == bsa.BSA_ERR_DEVICE and flags == 2, (code, flags)


# ------------------------------------------------------------ norm + rotation

def _qkv(B, N, Hq, Hkv, d, dtype, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g) * torch.exp(
        spread * torch.randn((B, N, Hq + 2 * Hkv, 1), generator=g))
    return x.to(dtype)


def _rope_inputs(rot, layout, scale=1.0):
    return (None if layout == "none" else
            500000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)), scale


def _weights(d, dtype, on, seed=5):
    if not on:
        return None, None
    g = torch.Generator().manual_seed(seed)
    return tuple((1 + 0.3 * torch.randn(d, generator=g)).to(dtype) for _ in range(2))


def _double(t):
    return None if t is None else t.double()


def _cuda(t):
    return None if t is None else t.cuda()


LAYOUT = {"none": 0, "half": 1, "pairs": 2}


def _encode_step(pipe, qkv, Hq, Hkv, w, freq, layout, pos, scale, eps=1e-5):
    return pipe.QkvStep(qkv, Hq, Hkv, q_weight=_cuda(w[0]), k_weight=_cuda(w[1]), eps=eps, inv_freq=_cuda(freq),
                        layout=LAYOUT[layout], positions=_cuda(pos), rope_scale=scale)


# B, N, Hq, Hkv, d, rot
ENCODE_SHAPES = [(1, 1, 1, 1, 128, 128), (3, 1, 32, 8, 128, 64), (2, 17, 4, 2, 64, 64), (1, 130, 7, 1, 128, 32),
                 (2, 5, 3, 3, 8, 8), (1, 33, 2, 1, 96, 96), (1, 19, 2, 1, 256, 128), (2, 9, 14, 2, 80, 40),
                 (1, 300, 28, 4, 128, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["none", "half", "pairs"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", ENCODE_SHAPES)
def test_encode(pipe, B, N, Hq, Hkv, d, rot, norm, layout, dtype):
    qkv = _qkv(B, N, Hq, Hkv, d, dtype)
    w = _weights(d, dtype, norm)
    freq, scale = _rope_inputs(rot, layout, 1.25)
    pos = torch.randint(-3, 1 << 20, (B, N), generator=torch.Generator().manual_seed(1)).int()
    step = _encode_step(pipe, qkv.cuda(), Hq, Hkv, w, freq, layout, pos, scale)
    got = step.run()
    want = plain.encode(qkv.double(), Hq, Hkv, _double(w[0]), _double(w[1]), 1e-5, freq, layout, pos, scale)
    for name, x in zip(("q", "k"), want[:2]):
        # one rounding to the type; before it fp32: the mean of d squares (d/16 + 8 sums), rsqrt, two products, an
        # angle to 2^-23 and two products of the pair: under 2^-19 of the row's largest value (twice, for a pair)
        top = x.abs().amax(-1, keepdim=True) * 2
        err = (got[name].cpu().double() - x).abs()
        assert bool((err <= HALF[dtype] * x.abs() + 2.0 ** -19 * top).all()), (name, (err / top).max())
    assert torch.equal(got["v"].cpu(), qkv[:, :, Hq + Hkv:].transpose(1, 2))


def test_encode_far_positions_and_default_positions(pipe):
    # positions at the ends of int32 keep their angle to the fixed point's precision: the frequency's 2^-53 in turns
    # times 2^31 positions is 2^-22 turns, 2^-19 rad
    qkv = _qkv(1, 4, 1, 1, 128, torch.float32, spread=0.0)
    freq, _ = _rope_inputs(128, "half")
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 12345678]], dtype=torch.int32)
    got = _encode_step(pipe, qkv.cuda(), 1, 1, (None, None), freq, "half", pos, 1.0).run()
    want = plain.encode(qkv.double(), 1, 1, None, None, 0, freq, "half", pos, 1.0)
    for name, x in zip(("q", "k"), want):
        assert (got[name].cpu().double() - x).abs().max() <= 2.0 ** -18 * 2 * x.abs().max()
    got = _encode_step(pipe, qkv.cuda(), 1, 1, (None, None), freq, "half", None, 1.0).run()["q"].clone()
    same = _encode_step(pipe, qkv.cuda(), 1, 1, (None, None), freq, "half", torch.arange(4).view(1, 4).int(),
                        1.0).run()["q"]
    assert torch.equal(got, same)


def test_encode_takes_a_slice_of_wider_rows_and_another_stream(pipe):
    wide = _qkv(2, 11, 5, 4, 64, torch.bfloat16).cuda()          # 13 heads a token
    part = wide[:, :, 2:10]                                       # 4 + 2 + 2 of them
    w = _weights(64, torch.bfloat16, True)
    freq, _ = _rope_inputs(64, "half")
    dense = _encode_step(pipe, part.contiguous(), 4, 2, w, freq, "half", None, 1.0)
    want = {n: t.clone() for n, t in dense.run().items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    step = _encode_step(pipe, part, 4, 2, w, freq, "half", None, 1.0)
    torch.cuda.synchronize()
    got = step.run(stream=stream)
    stream.synchronize()
    for n in ("q", "k", "v"):
        assert torch.equal(got[n], want[n])
    with pytest.raises(ValueError):
        _encode_step(pipe, wide[:, :, ::2][:, :, :6], 2, 2, w, freq, "half", None, 1.0).run()


def test_encode_rows_of_zeros_infinities_and_nan_stay_apart(pipe):
    qkv = _qkv(1, 6, 2, 1, 64, torch.float32)
    qkv[0, 1] = 0.0
    qkv[0, 3, 0, 5] = math.inf
    qkv[0, 4, 0, 7] = math.nan
    w = _weights(64, torch.float32, True)
    freq, _ = _rope_inputs(32, "pairs")
    got = _encode_step(pipe, qkv.cuda(), 2, 1, w, freq, "pairs", None, 1.0).run()
    assert bool((got["q"][0, :, 1] == 0).all()) and bool((got["k"][0, :, 1] == 0).all())
    bad = ~torch.isfinite(got["q"]).all(-1)[0].cpu()
    assert bad[0].tolist() == [False, False, False, True, True, False] and not bad[1].any()
    # without a norm, channels that are not rotated pass as they are
    got = _encode_step(pipe, qkv.cuda(), 2, 1, (None, None), freq, "pairs", None, 1.0).run()
    assert torch.equal(got["q"][..., 32:].cpu(), qkv[:, :, :2, 32:].transpose(1, 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["none", "half", "pairs"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", ENCODE_SHAPES)
def test_encode_backward(pipe, B, N, Hq, Hkv, d, rot, norm, layout, dtype):
    qkv = _qkv(B, N, Hq, Hkv, d, dtype, spread=1.0)
    w = _weights(d, dtype, norm)
    freq, scale = _rope_inputs(rot, layout, 0.75)
    g = torch.Generator().manual_seed(2)
    pos = torch.randint(-3, 1 << 20, (B, N), generator=g).int()
    grads = [torch.randn((B, h, N, d), generator=g) for h in (Hq, Hkv, Hkv)]
    step = _encode_step(pipe, qkv.cuda(), Hq, Hkv, w, freq, layout, pos, scale)
    got = step.backward(*(x.cuda() for x in grads))
    want, (size, dw_size) = plain.encode_grad(qkv.double(), Hq, Hkv, _double(w[0]), _double(w[1]), 1e-5, freq, layout,
                                              pos, scale, *(x.double() for x in grads))
    # as the forward, over the sizes of the terms: two sums of d products, about 30 roundings on the longest way
    err = (got["d_qkv"].cpu().double() - want[0]).abs()
    assert bool((err <= HALF[dtype] * want[0].abs() + 2.0 ** -18 * size).all()), (err / (size + 1e-30)).max()
    if norm:
        rows = B * N * max(Hq, Hkv)
        for name, x, s in zip(("d_q_weight", "d_k_weight"), want[1:], dw_size):
            # at most `rows` terms on one lane's way, each 2^-20 off, then 32 groups
            err = (got[name].cpu().double() - x).abs()
            assert bool((err <= ((rows + 32) * 2.0 ** -24 + 2.0 ** -20) * s).all())
        again = {n: got[n].clone() for n in ("d_qkv", "d_q_weight", "d_k_weight")}
        step.backward(*(x.cuda() for x in grads))
        assert all(torch.equal(again[n], got[n]) for n in again)


@pytest.mark.parametrize("exponent", [-45, -20, 30])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_encode_and_backward_of_tiny_and_large_rows_without_eps(pipe, exponent, dtype):
    # the norm does not see a factor on a row; its gradient is divided by it (2^45: the cube of 1/rms leaves fp32)
    qkv = _qkv(1, 21, 4, 2, 128, dtype, spread=0.0) * 2.0 ** exponent
    w = _weights(128, dtype, True)
    freq, _ = _rope_inputs(128, "half")
    g = torch.Generator().manual_seed(4)
    grads = [torch.randn((1, h, 21, 128), generator=g) for h in (4, 2, 2)]
    step = _encode_step(pipe, qkv.cuda(), 4, 2, w, freq, "half", None, 1.0, eps=0.0)
    out = step.run()
    wd = [x.double() for x in w]
    for name, x in zip(("q", "k"), plain.encode(qkv.double(), 4, 2, *wd, 0.0, freq, "half", None, 1.0)[:2]):
        top = x.abs().amax(-1, keepdim=True) * 2
        assert bool(((out[name].cpu().double() - x).abs() <= HALF[dtype] * x.abs() + 2.0 ** -19 * top).all()), name
    got = step.backward(*(x.cuda() for x in grads))
    want, (size, _) = plain.encode_grad(qkv.double(), 4, 2, *wd, 0.0, freq, "half", None, 1.0,
                                        *(x.double() for x in grads))
    err = (got["d_qkv"].cpu().double() - want[0]).abs()
    assert bool((err <= HALF[dtype] * want[0].abs() + 2.0 ** -18 * size).all()), (err / (size + 1e-30)).max()


def test_encode_backward_agrees_with_differences_of_the_kernel(pipe):
    # fp32, a directional difference of the forward kernel itself
    B, N, Hq, Hkv, d = 1, 13, 4, 2, 64
    qkv = _qkv(B, N, Hq, Hkv, d, torch.float32, spread=0.3)
    w = _weights(d, torch.float32, True)
    freq, _ = _rope_inputs(64, "half")
    g = torch.Generator().manual_seed(3)
    grads = [torch.randn((B, h, N, d), generator=g) for h in (Hq, Hkv, Hkv)]
    got = _encode_step(pipe, qkv.cuda(), Hq, Hkv, w, freq, "half", None, 1.0).backward(*(x.cuda() for x in grads))
    way = torch.randn(qkv.shape, generator=g)
    wway = [torch.randn(d, generator=g) for _ in range(2)]
    h, sides = 2.0 ** -7, []
    for sign in (1, -1):
        out = _encode_step(pipe, (qkv + sign * h * way).cuda(), Hq, Hkv,
                           tuple(a + sign * h * b for a, b in zip(w, wway)), freq, "half", None, 1.0).run()
        sides.append(sum((out[n].cpu().double() * x.double()).sum() for n, x in zip(("q", "k", "v"), grads)))
    slope = ((sides[0] - sides[1]) / (2 * h)).item()
    want = (got["d_qkv"].cpu().double() * way.double()).sum() + sum(
        (got[n].cpu().double() * x.double()).sum() for n, x in zip(("d_q_weight", "d_k_weight"), wway))
    # the curve's third derivative times h^2/6: h^2 = 6e-5, terms of size 1 on sqrt(rows d) = 75 random ones
    assert abs(slope - want.item()) <= 0.02 * math.sqrt(qkv.numel()) * 0.1 + 1e-3 * abs(slope)


# ------------------------------------------------------------ quantised cache

def _pools(pages, Hkv, d, seed=0):
    """Pools of random bytes: whatever a page held before."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)  # noqa: E731
    return r(pages, Hkv, 64, d), r(pages, Hkv, 64, d), r(pages, Hkv, 64), r(pages, Hkv, 64)


def _rows_like(g, *shape):
    return (torch.randn(shape, generator=g) * torch.exp(2 * torch.randn(shape[:-1] + (1,), generator=g))).bfloat16()


# d, T, lens (tokens held before)
APPENDS = [(128, 1, [0, 63, 64, 127]), (128, 65, [0, 1, 63, 64]), (64, 200, [0, 31, 64, 100]), (8, 3, [62, 61, 0, 64]),
           (96, 130, [5, 0, 64, 63]), (256, 67, [0, 60, 61, 64])]


@pytest.mark.parametrize("d,T,lens", APPENDS)
@pytest.mark.parametrize("ragged", [False, True])
def test_append_and_read_back(bsa, d, T, lens, ragged):
    B, Hkv, nb = len(lens), 3, 6
    g = torch.Generator().manual_seed(d + T)
    pages = B * nb + 2
    host = _pools(pages, Hkv, d)
    dev = [t.cuda() for t in host]
    table = torch.randperm(pages, generator=g)[:B * nb].view(B, nb).int()
    lens_t = torch.tensor(lens, dtype=torch.int32)
    # what the sequences hold already is well formed
    for b, n in enumerate(lens):
        for t in range(n):
            p, o = table[b, t // 64], t % 64
            for kv in (0, 1):
                c, e = plain.quantise(_rows_like(g, Hkv, d).double().numpy())
                host[kv][p, :, o], host[2 + kv][p, :, o] = torch.from_numpy(c), torch.from_numpy(e)
    for a, b in zip(dev, host):
        a.copy_(b)
    k_new, v_new = _rows_like(g, B, Hkv, T, d), _rows_like(g, B, Hkv, T, d)
    k_new[0, 0, 0] = 0.0
    k_new[1, 0, 0, 3], v_new[1, 0, 0, :2] = math.inf, torch.tensor([math.nan, -math.inf])
    k_new[2, 1, 0, 1], v_new[2, 1, 0, 0] = 3e38, 1e-40        # the exponent's upper and lower ends
    new = [max(0, T - 2 * b) for b in range(B)] if ragged else [T] * B
    pooled = torch.full((B, Hkv, nb, d), -7.0, device="cuda")
    shape = bsa.make_shape(B, Hkv, Hkv, T, nb * 64, d, 64, torch.bfloat16)
    bsa.bsa_paged_append_quant(shape, k_new.cuda(), v_new.cuda(), lens_t.cuda(), table.cuda(), *dev, pooled,
                               new_lens=torch.tensor(new, dtype=torch.int32).cuda() if ragged else None)
    want_pool = torch.full((B, Hkv, nb, d), -7.0)
    for kv, x in enumerate((k_new, v_new)):
        c, e = plain.quantise(x.double().numpy())
        for b in range(B):
            for t in range(new[b]):
                p, o = table[b, (lens[b] + t) // 64], (lens[b] + t) % 64
                host[kv][p, :, o], host[2 + kv][p, :, o] = torch.from_numpy(c[b, :, t]), torch.from_numpy(e[b, :, t])
    for a, b in zip(dev, host):
        assert torch.equal(a.cpu(), b)                        # the new rows, and every other byte as it was
    for b in range(B):
        for j in range(lens[b] // 64, (lens[b] + new[b]) // 64):
            p = table[b, j]
            keys = plain.dequantise(host[0][p].numpy(), host[2][p].numpy()).astype(np.float32)   # exact in fp32
            total = np.zeros((Hkv, d), np.float32)
            for t in range(64):
                total = total + keys[:, t]
            want_pool[b, :, j] = torch.from_numpy(total / np.float32(64))
    got = pooled.cpu()
    assert torch.equal(torch.nan_to_num(got, 99.0), torch.nan_to_num(want_pool, 99.0))
    # read back: exact, rows past the sequences untouched
    held = (lens_t + torch.tensor(new)).int()
    starts = torch.tensor([0, 1, 63, 64], dtype=torch.int32)
    for dtype, with_starts in ((torch.bfloat16, False), (torch.float32, True)):
        R = 70
        outs = [torch.full((B, Hkv, R, d), 5.0, dtype=dtype, device="cuda") for _ in range(2)]
        rshape = bsa.make_shape(B, Hkv, Hkv, R, nb * 64, d, 64, dtype)
        bsa.bsa_paged_read_quant(rshape, *dev, table.cuda(), held.cuda(), *outs,
                                 starts=starts.cuda() if with_starts else None)
        for kv in (0, 1):
            want = torch.full((B, Hkv, R, d), 5.0, dtype=torch.float64)
            for b in range(B):
                for t in range(R):
                    at = t + (int(starts[b]) if with_starts else 0)
                    if at < held[b]:
                        p, o = table[b, at // 64], at % 64
                        want[b, :, t] = torch.from_numpy(plain.dequantise(host[kv][p, :, o].numpy(),
                                                                          host[2 + kv][p, :, o].numpy()))
            assert torch.equal(torch.nan_to_num(outs[kv].cpu().double(), 99.0), torch.nan_to_num(want, 99.0))
    only = torch.full_like(outs[1], 5.0)
    bsa.bsa_paged_read_quant(rshape, *dev, table.cuda(), held.cuda(), None, only, starts=starts.cuda())
    assert torch.equal(torch.nan_to_num(only, 99.0), torch.nan_to_num(outs[1], 99.0))


def test_appends_token_by_token_are_one_append(bsa):
    B, Hkv, d, nb, T = 2, 2, 128, 3, 130
    g = torch.Generator().manual_seed(8)
    k, v = _rows_like(g, B, Hkv, T, d).cuda(), _rows_like(g, B, Hkv, T, d).cuda()
    table = torch.randperm(B * nb, generator=g).view(B, nb).int().cuda()
    sides = []
    for one_by_one in (False, True):
        pools = [t.cuda().zero_() for t in _pools(B * nb, Hkv, d)]
        pooled = torch.zeros((B, Hkv, nb, d), device="cuda")
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        for t0 in range(0, T, 1 if one_by_one else T):
            n = 1 if one_by_one else T
            shape = bsa.make_shape(B, Hkv, Hkv, n, nb * 64, d, 64, torch.bfloat16)
            bsa.bsa_paged_append_quant(shape, k[:, :, t0:t0 + n].contiguous(), v[:, :, t0:t0 + n].contiguous(), lens,
                                       table, *pools, pooled)
            lens += n
        sides.append(pools + [pooled])
    assert all(torch.equal(a, b) for a, b in zip(*sides))


def test_bad_pages_and_positions_are_flagged_and_skipped(bsa):
    B, Hkv, d, nb = 3, 2, 64, 2
    pools = [t.cuda() for t in _pools(4, Hkv, d)]
    before = [t.clone() for t in pools]
    g = torch.Generator().manual_seed(1)
    x = _rows_like(g, B, Hkv, 1, d).cuda()
    shape = bsa.make_shape(B, Hkv, Hkv, 1, nb * 64, d, 64, torch.bfloat16)
    # a page past the pools, a negative page, a position past the table, a negative length: each alone is flagged
    for table, lens in (([[0, 1], [4, 0], [2, 3]], [64, 3, 0]), ([[0, 1], [-1, 0], [2, 3]], [64, 3, 0]),
                        ([[0, 1], [2, 3], [2, 3]], [64, 128, 0]), ([[0, 1], [2, 3], [2, 3]], [64, -1, 0])):
        table = torch.tensor(table, dtype=torch.int32).cuda()
        lens = torch.tensor(lens, dtype=torch.int32).cuda()
        for a, b in zip(pools, before):
            a.copy_(b)
        bsa.bsa_paged_append_quant(shape, x, x, lens, table, *pools, None)
        _flagged(bsa)
        c, e = plain.quantise(x.cpu().double().numpy())
        want = before[0].clone()
        want[1, :, 0], want[2, :, 0] = torch.from_numpy(c[0, :, 0]).cuda(), torch.from_numpy(c[2, :, 0]).cuda()
        assert torch.equal(pools[0], want)
        if int(lens[1]) == 3:
            out = torch.full((B, Hkv, 1, d), 5.0, dtype=torch.bfloat16, device="cuda")
            bsa.bsa_paged_read_quant(shape, *before, table, torch.full_like(lens, 128), out, None)
            _flagged(bsa)
            assert bool((out[1] == 5).all()) and not bool((out[0] == 5).all())


# --------------------------------------------------------------------- decode

def _cache(lens, Hkv, d, nb, seed=0, spread=1.0):
    """Pools of NaN codes and exponent 255 with the sequences' rows written where the table says; table entries
    behind a sequence are -1."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = B * nb + 3
    pools = [np.full((pages, Hkv, 64, d), 127, np.uint8) for _ in range(2)]
    exps = [np.full((pages, Hkv, 64), 255, np.uint8) for _ in range(2)]
    table = torch.randperm(pages, generator=g)[:B * nb].view(B, nb).int().numpy()
    r = np.random.default_rng(seed)
    for b, n in enumerate(lens):
        used = -(-n // 64)
        for j in range(used):
            m = min(64, n - 64 * j)
            for kv in range(2):
                pools[kv][table[b, j], :, :m] = r.integers(0, 127, (Hkv, m, d)) | (r.integers(0, 2, (Hkv, m, d)) << 7)
                exps[kv][table[b, j], :, :m] = np.clip(np.round(117 + spread * r.standard_normal((Hkv, m))), 10, 246)
        table[b, used:] = -1
    return pools[0], pools[1], exps[0], exps[1], table


def _check_decode(bsa, q, cache, lens, idx, scale=None, what="", far=0.0, least=0.0):
    B, Hq, d = q.shape
    k, v, ke, ve, table = cache
    Hkv, nb = k.shape[1], table.shape[1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    shape = bsa.make_shape(B, Hq, Hkv, 1, nb * 64, d, 64, torch.bfloat16)
    stride = 0 if idx is None else idx.shape[-1]
    ws = torch.full((bsa.bsa_workspace_bytes(bsa.BSA_OP_DECODE_QUANT, shape, stride),), 255, dtype=torch.uint8,
                    device="cuda")
    o = torch.full((B, Hq, d), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq), math.nan, device="cuda")
    args = [torch.from_numpy(x).cuda() for x in (k, v, ke, ve, table)]
    bsa.bsa_sparse_attn_decode_quant(shape, q.cuda(), *args, torch.tensor(lens, dtype=torch.int32).cuda(),
                                     None if idx is None else torch.from_numpy(idx).cuda(), stride, scale, ws, o, lse)
    torch.cuda.synchronize()
    want, want_lse, weight, size = plain.decode(q.double().numpy(), k, v, ke, ve, table, lens, idx, scale)
    got, got_lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    # a logit is a sum of d products in fp32, d 2^-24 of the products' sizes (taken whole, whichever way the matrix
    # unit adds); a weight moves by that, its fp16 rounding (2^-11) and the exponential (2^-22); the output is rounded
    # once more
    off = size * d * 2.0 ** -24 * 2 + 2.0 ** -20 + far
    tol = HALF[torch.bfloat16] * np.abs(want) + (2.0 ** -11 + 2 * off)[..., None] * 1.01 * weight + least
    err = np.abs(got - want)
    assert np.all(err <= tol), (what, np.unravel_index(np.argmax(err - tol), err.shape), (err - tol).max())
    none = np.isinf(want_lse)
    assert np.array_equal(none, np.isinf(got_lse) & (got_lse < 0)), what
    assert np.all(got[none] == 0)
    lse_off = np.abs(got_lse[~none] - want_lse[~none])
    assert np.all(lse_off <= (off[~none] + 2.0 ** -22 * (4 + np.abs(want_lse[~none])))), what
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 1), (14, 2), (16, 2), (9, 1), (32, 2), (6, 6)])
def test_decode_every_block(bsa, Hq, Hkv, d):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 128, 300]
    q = torch.randn((len(lens), Hq, d), generator=torch.Generator().manual_seed(Hq)).bfloat16()
    _check_decode(bsa, q, _cache(lens, Hkv, d, 5), lens, None)


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (28, 4), (16, 1)])
def test_decode_kept_blocks(bsa, Hq, Hkv):
    lens = [700, 1, 64, 0, 449, 130]
    B, nb, d = len(lens), 11, 128
    r = np.random.default_rng(4)
    idx = np.full((B, Hkv, 6), -1, np.int32)
    for b, n in enumerate(lens):
        own = -(-n // 64)
        for g in range(Hkv):
            kept = np.sort(r.permutation(max(own - 1, 0))[:4])
            kept = np.append(kept, own - 1) if own else kept
            idx[b, g, :len(kept)] = kept
    q = torch.randn((B, Hq, d), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = _cache(lens, Hkv, d, nb, seed=2)
    _check_decode(bsa, q, cache, lens, idx)
    # the contract's corners: holes, a block twice, blocks past the sequence's own length, no block at all
    idx[0, 0] = [-1, 3, -1, 3, 10, 0]
    idx[1, 0] = [-1, -1, -1, -1, -1, 0]
    idx[2, 0] = [1, 2, 10, -1, -1, -1]
    idx[4, 0] = -1
    _check_decode(bsa, q, cache, lens, idx)


@pytest.mark.parametrize("splits", [0, 1, 7, 61, 1000])
def test_decode_with_other_splits(bsa, splits):
    lens = [1500, 3, 0, 64, 777]
    q = torch.randn((5, 8, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    prev = bsa.bsa_decode_split_override(splits)
    try:
        _check_decode(bsa, q, _cache(lens, 2, 128, 24), lens, None)
    finally:
        bsa.bsa_decode_split_override(prev)


@pytest.mark.parametrize("B,Hkv,G", [(20, 8, 4), (40, 8, 1), (80, 8, 3), (20, 8, 12), (40, 8, 16),
                                     (16, 8, 4), (30, 8, 2), (64, 8, 1), (16, 8, 9), (64, 8, 10)])
def test_decode_of_many_rows(bsa, B, Hkv, G):
    """About as many rows as multiprocessors, and more: blocks of threads split into teams, ranges that hold whole rows
    (then one launch writes every output, those of rows without a block too), ranges with several rows each."""
    r = np.random.default_rng(B + G)
    lens = r.integers(0, 260, B).tolist()
    nb, keep = 5, 3
    q = torch.randn((B, Hkv * G, 64), generator=torch.Generator().manual_seed(G)).bfloat16()
    cache = _cache(lens, Hkv, 64, nb, seed=B)
    _check_decode(bsa, q, cache, lens, None)
    idx = np.full((B, Hkv, keep), -1, np.int32)
    for b, n in enumerate(lens):
        own = -(-n // 64)
        for g in range(Hkv):
            kept = np.sort(r.permutation(own)[:keep])
            idx[b, g, :len(kept)] = kept
    idx[1, 0] = -1
    idx[2, 1] = [-1, -2 ** 31, -1]
    _check_decode(bsa, q, cache, lens, idx)


@pytest.mark.parametrize("B,Hkv,G,d", [(12, 8, 4, 128), (11, 8, 12, 128), (9, 9, 16, 64), (18, 8, 9, 128), (3, 4, 16, 128),
                                       (37, 2, 1, 64)])
def test_decode_every_block_of_rows_cut_by_ranges(bsa, B, Hkv, G, d):
    """Rows of lengths from none to 30 blocks, cut between teams of 3 to 16 warps; a range holds parts of several rows."""
    r = np.random.default_rng(B * G)
    lens = r.integers(0, 1900, B).tolist()
    lens[1], lens[-1] = 0, 1920
    q = torch.randn((B, Hkv * G, d), generator=torch.Generator().manual_seed(B)).bfloat16()
    _check_decode(bsa, q, _cache(lens, Hkv, d, 30, seed=G), lens, None)


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [0] * 200])
def test_decode_of_empty_sequences_alone(bsa, lens):
    q = torch.randn((len(lens), 8, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    cache = _cache(lens, 2, 128, 3)
    _check_decode(bsa, q, cache, lens, None)
    _check_decode(bsa, q, cache, lens, np.zeros((len(lens), 2, 2), np.int32))


@pytest.mark.parametrize("G", [2, 16])
def test_decode_of_the_largest_batch(bsa, G):
    lens = [0] * 8192
    for b in range(0, 8192, 37):
        lens[b] = 1 + b % 100
    lens[8191] = 128
    q = torch.randn((8192, G, 64), generator=torch.Generator().manual_seed(G)).bfloat16()
    _check_decode(bsa, q, _cache(lens, 1, 64, 2), lens, None)


@pytest.mark.parametrize("spread,gain", [(0.0, 30.0), (12.0, 1.0), (0.0, 0.0), (4.0, 1e-30), (3.0, 1e4)])
def test_decode_steep_flat_and_uneven_rows(bsa, spread, gain):
    # large logits, exponents far apart (values 2^12 apart and more), zero and tiny queries
    lens = [500, 33]
    q = (gain * torch.randn((2, 4, 128), generator=torch.Generator().manual_seed(6))).bfloat16()
    _check_decode(bsa, q, _cache(lens, 1, 128, 9, seed=3, spread=spread), lens, None,
                  scale=1 / math.sqrt(128) / max(1.0, gain / 30) / 2.0 ** (2 * spread))


@pytest.mark.parametrize("zeros", ["all", "before", "behind", "between", "one"])
@pytest.mark.parametrize("e_rest", [60, 119, 165, 240])
def test_decode_with_rows_of_zero_values(bsa, zeros, e_rest):
    """A value row of zeros (exponent 10) has the weight of its logit, whatever stands beside it: in long runs before,
    behind or between other rows, whose exponents differ from its own by up to 230."""
    lens = [2500, 40, 700]
    cache = _cache(lens, 1, 128, 40, seed=5)
    r = np.random.default_rng(5)
    for b, n in enumerate(lens):
        t = np.arange(n)
        off = {"all": t >= 0, "before": t < n - 3, "behind": t > 2, "between": r.random(n) < 0.5, "one": t == n // 2}[zeros]
        page = cache[4][b, t // 64]
        cache[1][page[off], 0, t[off] % 64] = 0
        cache[3][page, 0, t % 64] = np.where(off, 10, e_rest)
    q = torch.randn((3, 8, 128), generator=torch.Generator().manual_seed(8)).bfloat16()
    # a logit against the reference, up to 128 octaves away: a rounding of 2^-18 octaves, three of them
    _check_decode(bsa, q, cache, lens, None, scale=0.02, far=3 * 2.0 ** -18)
    idx = np.full((3, 1, 4), -1, np.int32)
    idx[0, 0], idx[1, 0, :1], idx[2, 0, :3] = [0, 7, 38, 39], [0], [0, 5, 10]
    _check_decode(bsa, q, cache, lens, idx, scale=0.02, far=3 * 2.0 ** -18)


@pytest.mark.parametrize("lo,hi", [(56, 60), (10, 20), (10, 90), (30, 246)])
def test_decode_of_tiny_values(bsa, lo, hi):
    # rows under exponent 56 (values under 2^-62) are off by at most 2^-94, absolute; their logits count in full
    lens = [900, 17]
    cache = _cache(lens, 2, 64, 15, seed=6)
    r = np.random.default_rng(lo)
    ve = np.where(cache[3] == 255, 255, r.integers(lo, hi + 1, cache[3].shape)).astype(np.uint8)
    q = torch.randn((2, 8, 64), generator=torch.Generator().manual_seed(10)).bfloat16()
    _check_decode(bsa, q, (*cache[:3], ve, cache[4]), lens, None, scale=0.02, far=3 * 2.0 ** -18,
                  least=2.0 ** -94)


def test_decode_ascending_logits_move_the_reference(bsa):
    # every 16 keys the largest logit grows by some 40: the running reference has to follow
    n, d = 640, 64
    cache = _cache([n], 1, d, 10)
    k = np.full_like(cache[0], 127)
    q = torch.zeros((1, 3, d))
    q[0, :, 0] = torch.tensor([1.0, -1.0, 0.125])
    k[cache[4][0]] = 0
    for t in range(n):
        k[cache[4][0, t // 64], 0, t % 64, 0] = min(126, 56 + t // 16)
    ke = np.where(cache[2] == 255, 255, 127).astype(np.uint8)
    _check_decode(bsa, q.bfloat16(), (k, cache[1], ke, cache[3], cache[4]), [n], None, scale=1.0)


def test_decode_nan_in_a_seen_row_shows_and_in_an_unseen_one_does_not(bsa):
    lens = [70]
    q = torch.randn((1, 4, 128), generator=torch.Generator().manual_seed(7)).bfloat16()
    cache = _cache(lens, 2, 128, 2)
    _check_decode(bsa, q, cache, lens, None)                    # rows past 70 hold NaN already
    shape = bsa.make_shape(1, 4, 2, 1, 128, 128, 64, torch.bfloat16)
    for pool, n in ((0, 70), (1, 70), (0, 1)):
        k = [x.copy() for x in cache]
        k[pool][k[4][0, 0], 0, 0, 5] = 127
        dev = [torch.from_numpy(x).cuda() for x in k]
        ws = torch.empty((bsa.bsa_workspace_bytes(bsa.BSA_OP_DECODE_QUANT, shape, 0),), dtype=torch.uint8,
                         device="cuda")
        o = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda")
        bsa.bsa_sparse_attn_decode_quant(shape, q.cuda(), *dev, torch.tensor([n], dtype=torch.int32).cuda(), None, 0,
                                         0.1, ws, o)
        bad = torch.isnan(o[0]).cpu()
        assert not bad[2:].any()
        assert bad[:2, 5].all() and (pool == 1 or bad[:2].all())
        assert pool == 0 or bad[:2].sum() == 2


def test_decode_flags_bad_blocks_and_pages(bsa):
    lens = [200, 200]
    q = torch.randn((2, 4, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    k, v, ke, ve, table = _cache(lens, 1, 128, 4)
    idx = np.array([[[0, 4, 3]], [[1, 2, -1]]], np.int32)       # block 4 of 4
    clean = idx.copy()
    clean[0, 0, 1] = -1
    want = plain.decode(q.double().numpy(), k, v, ke, ve, table, lens, clean, 0.1)[0]
    shape = bsa.make_shape(2, 4, 1, 1, 256, 128, 64, torch.bfloat16)
    ws = torch.empty((bsa.bsa_workspace_bytes(bsa.BSA_OP_DECODE_QUANT, shape, 3),), dtype=torch.uint8, device="cuda")
    for case in ("block", "page", "negative page"):
        t, i = table.copy(), idx.copy()
        if case != "block":
            i[0, 0, 1] = 2
            t[0, 2] = len(k) if case == "page" else -5
        o = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
        bsa.bsa_sparse_attn_decode_quant(shape, q.cuda(), *(torch.from_numpy(x).cuda() for x in (k, v, ke, ve, t)),
                                         torch.tensor(lens, dtype=torch.int32).cuda(), torch.from_numpy(i).cuda(), 3,
                                         0.1, ws, o)
        _flagged(bsa)
        assert np.abs(o.cpu().double().numpy() - want).max() <= 2.0 ** -7 * np.abs(want).max()


def test_decode_lengths_are_taken_within_the_table(bsa):
    lens = [128]
    q = torch.randn((1, 4, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    cache = _cache(lens, 1, 128, 2)
    shape = bsa.make_shape(1, 4, 1, 1, 128, 128, 64, torch.bfloat16)
    dev = [torch.from_numpy(x).cuda() for x in cache]
    ws = torch.empty((bsa.bsa_workspace_bytes(bsa.BSA_OP_DECODE_QUANT, shape, 0),), dtype=torch.uint8, device="cuda")
    outs = []
    for n in (128, None, 1000, -4):
        o = torch.full((1, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        bsa.bsa_sparse_attn_decode_quant(shape, q.cuda(), *dev,
                                         None if n is None else torch.tensor([n], dtype=torch.int32).cuda(), None, 0,
                                         0.1, ws, o)
        outs.append(o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and bool((outs[3] == 0).all())


def test_decode_pages_past_32_bits(bsa):
    # the last pages of pools of more than 2^31 bytes
    pages, Hkv, d = 33000, 8, 128
    cache = _cache([130], Hkv, d, 3)
    big = [torch.zeros((pages, Hkv, 64, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    exps = [torch.zeros((pages, Hkv, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    n = cache[0].shape[0]
    for dst, src in zip(big + exps, cache):
        dst[pages - n:] = torch.from_numpy(src).cuda()
    table = torch.from_numpy(np.where(cache[4] >= 0, cache[4] + pages - n, -1).astype(np.int32)).cuda()
    q = torch.randn((1, 8, d), generator=torch.Generator().manual_seed(2)).bfloat16()
    shape = bsa.make_shape(1, 8, Hkv, 1, 192, d, 64, torch.bfloat16)
    lens = torch.tensor([130], dtype=torch.int32).cuda()
    ws = torch.empty((bsa.bsa_workspace_bytes(bsa.BSA_OP_DECODE_QUANT, shape, 0),), dtype=torch.uint8, device="cuda")
    o, small = (torch.zeros((1, 8, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bsa.bsa_sparse_attn_decode_quant(shape, q.cuda(), *big, *exps, table, lens, None, 0, 0.1, ws, o)
    bsa.bsa_sparse_attn_decode_quant(shape, q.cuda(), *(torch.from_numpy(x).cuda() for x in cache), lens, None, 0, 0.1,
                                     ws, small)
    assert torch.equal(o, small) and bool((o != 0).any())
    rows = [torch.zeros((1, Hkv, 130, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bsa.bsa_paged_read_quant(bsa.make_shape(1, Hkv, Hkv, 130, 192, d, 64, torch.bfloat16), *big, *exps, table, lens,
                             *rows)
    x = torch.from_numpy(plain.dequantise(cache[0][cache[4][0, 2], :, 1], cache[2][cache[4][0, 2], :, 1]))
    assert torch.equal(rows[0][0, :, 129].cpu().double(), x)
    new = _rows_like(torch.Generator().manual_seed(3), 1, Hkv, 1, d).cuda()
    bsa.bsa_paged_append_quant(bsa.make_shape(1, Hkv, Hkv, 1, 192, d, 64, torch.bfloat16), new, new, lens, table, *big,
                               *exps)
    c, e = plain.quantise(new.cpu().double().numpy())
    at = int(table[0, 2])
    assert torch.equal(big[1][at, :, 2].cpu(), torch.from_numpy(c[0, :, 0]))
    assert torch.equal(exps[0][at, :, 2].cpu(), torch.from_numpy(e[0, :, 0]))


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("ncols", [1, 2, 31, 300, 512, 513, 1024, 1025, 2048, 2049, 4097, 8192])
def test_select_by_length(bsa, ncols):
    r = np.random.default_rng(ncols)
    per, block = 3, 64
    lens = [0, 1, 64, 65, ncols * 64, max(1, ncols * 64 - 63), max(1, ncols * 32 + 5)]
    rows = per * len(lens)
    for kb in (0, 1, 7, 300):
        s = r.integers(-4, 5, (rows, ncols)).astype(np.float32)
        s[0::4, ::3] = np.nan
        s[1::4, ::2] = -np.inf
        s[2::4] = 0.0
        for seq, n in enumerate(lens):                           # columns that are not candidates are not read
            s[seq * per:(seq + 1) * per, max(0, -(-n // block) - 1):] = np.inf
        stride = kb + 3
        want, cnt = plain.select(s, lens, per, block, kb, stride)
        idx = torch.full((rows, stride), -7, dtype=torch.int32, device="cuda")
        count = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
        bsa.bsa_topk_select_lens(torch.from_numpy(s).cuda(), rows, ncols, torch.tensor(lens, dtype=torch.int32).cuda(),
                                 per, block, kb, idx, stride, count)
        assert np.array_equal(idx.cpu().numpy(), want), (ncols, kb)
        assert np.array_equal(count.cpu().numpy(), cnt)
        if max(lens) > ncols * 64:       # 65 tokens where the row has one column: taken as one block, and flagged
            _flagged(bsa)


@pytest.mark.parametrize("ncols", [40, 1000, 5000])
def test_select_by_length_of_close_tiny_and_huge_scores(bsa, ncols):
    """Scores that differ in their last bits, subnormals, both zeros, the largest and infinite ones, and many equal to
    the threshold: the order is the full fp32 one."""
    r = np.random.default_rng(ncols)
    tiny = np.float32(2.0 ** -149)
    rows = [np.float32(1.5) + np.arange(ncols, dtype=np.float32) % 7 * np.float32(2.0 ** -23),
            r.integers(-3, 4, ncols).astype(np.float32) * tiny,
            np.where(r.random(ncols) < 0.5, np.float32(-0.0), np.float32(0.0)),
            r.choice(np.array([np.inf, -np.inf, np.nan, 3.4e38, -3.4e38, 3.3e38, 1.0], np.float32), ncols),
            -np.exp(r.standard_normal(ncols) * 20).astype(np.float32),
            r.standard_normal(ncols).astype(np.float32),
            np.full(ncols, np.nan, np.float32),
            (r.integers(0, 2, ncols) * 2.0 ** -20 + 1).astype(np.float32)]
    s = np.stack([row[r.permutation(ncols)] for row in rows])
    lens = [64 * ncols] * len(rows)
    for kb in (1, 5, ncols // 3, ncols - 2):
        want, cnt = plain.select(s, lens, 1, 64, kb, kb + 1)
        idx = torch.full((len(rows), kb + 1), -7, dtype=torch.int32, device="cuda")
        count = torch.full((len(rows),), -7, dtype=torch.int32, device="cuda")
        bsa.bsa_topk_select_lens(torch.from_numpy(s).cuda(), len(rows), ncols,
                                 torch.tensor(lens, dtype=torch.int32).cuda(), 1, 64, kb, idx, kb + 1, count)
        for row in range(len(rows)):
            assert np.array_equal(idx[row].cpu().numpy(), want[row]), (ncols, kb, row)
        assert np.array_equal(count.cpu().numpy(), cnt)


def test_select_by_length_of_rows_at_an_odd_address(bsa):
    base = torch.randn(4 * 300 + 1, generator=torch.Generator().manual_seed(1)).cuda()
    s = base[1:].view(4, 300)
    idx = torch.zeros((4, 9), dtype=torch.int32, device="cuda")
    bsa.bsa_topk_select_lens(s, 4, 300, torch.tensor([300 * 64, 5000], dtype=torch.int32).cuda(), 2, 64, 8, idx, 9)
    want, _ = plain.select(s.cpu().numpy(), [300 * 64, 5000], 2, 64, 8, 9)
    assert np.array_equal(idx.cpu().numpy(), want)


def test_select_by_length_flags_what_the_table_cannot_hold(bsa):
    s = torch.randn((2, 5)).cuda()
    idx = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    bsa.bsa_topk_select_lens(s, 2, 5, torch.tensor([321, -3], dtype=torch.int32).cuda(), 1, 64, 2, idx, 3)
    _flagged(bsa)
    want, _ = plain.select(s.cpu().numpy(), [320, 0], 1, 64, 2, 3)
    assert np.array_equal(idx.cpu().numpy(), want)


# -------------------------------------------------------------------- together

def test_projection_prefill_and_both_backwards(bsa, pipe):
    """QkvStep -> gated PrefillStep -> its backward -> QkvStep's, against autograd in 64 bits of the same formulas on
    the kept blocks and gate scores that the step chose."""
    B, N, Hq, Hkv, d, block, kb = 1, 512, 4, 2, 128, 64, 3
    qkv = _qkv(B, N, Hq, Hkv, d, torch.bfloat16, spread=0.3)
    w = _weights(d, torch.bfloat16, True)
    freq, _ = _rope_inputs(128, "half")
    enc = _encode_step(pipe, qkv.cuda(), Hq, Hkv, w, freq, "half", None, 1.0)
    out = enc.run()
    step = pipe.PrefillStep(out["q"], out["k"], out["v"], block, kb, gated=False)
    step.run()
    d_o = torch.randn((B, Hq, N, d), generator=torch.Generator().manual_seed(4)).bfloat16()
    step.backward(d_o.cuda())
    got = enc.backward(step.bufs["dq"], step.bufs["dk"], step.bufs["dv"])
    idx = step.bufs["idx"].cpu()
    leaves = [qkv.double().requires_grad_(), w[0].double().requires_grad_(), w[1].double().requires_grad_()]
    q, k, v = plain.encode(leaves[0], Hq, Hkv, leaves[1], leaves[2], 1e-5, freq, "half", None, 1.0)
    seen = torch.zeros((B, Hkv, N, N), dtype=torch.bool)
    for g in range(Hkv):
        for i in range(N // block):
            for j in idx[0, g, i][idx[0, g, i] >= 0].tolist():
                seen[0, g, i * block:(i + 1) * block, j * block:(j + 1) * block] = True
    seen &= torch.ones((N, N), dtype=torch.bool).tril()
    G = Hq // Hkv
    x = q @ k.repeat_interleave(G, 1).transpose(2, 3) / math.sqrt(d)
    o = torch.softmax(x.masked_fill(~seen.repeat_interleave(G, 1), -math.inf), -1) @ v.repeat_interleave(G, 1)
    (o * d_o.double()).sum().backward()
    # q, k, v, P and dS are each rounded to bf16 (2^-8) on the way, averaged over many terms: in the 2-norm a few
    # roundings' worth
    for name, leaf in zip(("d_qkv", "d_q_weight", "d_k_weight"), leaves):
        rel = (got[name].cpu().double() - leaf.grad).norm() / leaf.grad.norm()
        assert rel <= 5 * 2.0 ** -8, (name, rel)
    rel = (step.bufs["o"].cpu().double() - o).norm() / o.norm()
    assert rel <= 3 * 2.0 ** -8


def test_ragged_serving_loop(bsa, pipe):
    """Prompts of different lengths appended from a padded projection, then tokens one by one: encode, append, select,
    attend; every step against the plain decode over the cache as it stands and the plain selection of its scores."""
    B, Hq, Hkv, d, nb, kb = 3, 8, 2, 128, 8, 2
    g = torch.Generator().manual_seed(11)
    freq, _ = _rope_inputs(128, "half")
    w = _weights(d, torch.bfloat16, True)
    pages = B * nb
    pools = [t.cuda() for t in _pools(pages, Hkv, d)]
    table = torch.randperm(pages, generator=g).view(B, nb).int().cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    step = pipe.QuantDecodeStep(q, *pools, table, lens, kb=kb)
    every = pipe.QuantDecodeStep(q, *pools, table, lens)
    prompt = torch.tensor([317, 64, 250], dtype=torch.int32)
    enc = _encode_step(pipe, _qkv(B, 320, Hq, Hkv, d, torch.bfloat16, spread=0.3).cuda(), Hq, Hkv, w, freq, "half",
                       None, 1.0)
    out = enc.run()
    step.append(out["k"], out["v"], new_lens=prompt.cuda())
    lens += prompt.cuda()
    for turn in range(6):
        pos = lens.clone().view(B, 1).cpu()
        tok = _encode_step(pipe, _qkv(B, 1, Hq, Hkv, d, torch.bfloat16, seed=20 + turn, spread=0.3).cuda(), Hq, Hkv, w,
                           freq, "half", pos, 1.0).run()
        step.append(tok["k"], tok["v"])
        lens += 1
        q.copy_(tok["q"][:, :, 0])
        step.run()
        every.run()
        torch.cuda.synchronize()
        host = [t.cpu().numpy() for t in pools] + [table.cpu().numpy()]
        n = lens.cpu().numpy()
        want_idx, want_cnt = plain.select(step.bufs["scores"].cpu().numpy().reshape(B * Hkv, nb), n, Hkv, 64, kb, kb + 1)
        assert np.array_equal(step.bufs["idx"].cpu().numpy().reshape(B * Hkv, -1), want_idx)
        assert np.array_equal(step.bufs["count"].cpu().numpy().reshape(-1), want_cnt)
        for s, idx in ((step, want_idx.reshape(B, Hkv, -1)), (every, None)):
            o, lse, weight, size = plain.decode(q.cpu().double().numpy(), *host, n, idx, 1 / math.sqrt(d))
            tol = HALF[torch.bfloat16] * np.abs(o) + (2.0 ** -10 + size * 2.0 ** -15)[..., None] * weight
            assert np.all(np.abs(s.bufs["o"].cpu().double().numpy() - o) <= tol)
            assert np.abs(s.bufs["lse"].cpu().double().numpy() - lse).max() <= 2.0 ** -14 * (1 + np.abs(lse).max())
    # the summary of every whole block is the mean of its stored keys
    for b in range(B):
        for j in range(int(lens[b]) // 64):
            p = int(table[b, j])
            keys = plain.dequantise(host[0][p], host[2][p])
            got = step.bufs["kbar"][b, :, j].cpu().double().numpy()
            assert np.abs(got - keys.mean(1)).max() <= 64 * 2.0 ** -24 * np.abs(keys).max()


def test_quantised_decode_of_a_cache_that_holds_bf16_values_is_the_paged_decode(bsa, pipe):
    """What is stored is exact in bf16: decoding the read-back rows from a bf16 paged cache gives the same attention."""
    B, Hq, Hkv, d, nb = 2, 8, 2, 128, 16
    g = torch.Generator().manual_seed(12)
    T = nb * 64
    pools = [t.cuda() for t in _pools(B * nb, Hkv, d)]
    table = torch.randperm(B * nb, generator=g).view(B, nb).int().cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.randn((B, Hq, d), generator=g).bfloat16().cuda()
    step = pipe.QuantDecodeStep(q, *pools, table, lens, kb=5)
    step.append(_rows_like(g, B, Hkv, T, d).cuda(), _rows_like(g, B, Hkv, T, d).cuda())
    lens += T
    k, v = (torch.empty((B, Hkv, T, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    step.read(k, v)
    step.run()
    other = pipe.DecodeStep(q, k, v, 64, 5)
    other.pool_cache()
    assert torch.equal(other.bufs["kbar"], step.bufs["kbar"])
    other.run()
    assert torch.equal(other.bufs["idx"], step.bufs["idx"])
    a, b = (s.bufs["o"].float() for s in (step, other))
    assert (a - b).norm() <= 2 * 2.0 ** -8 * b.norm()       # two roundings of o, and of bf16 and fp16 weights
    assert (step.bufs["lse"] - other.bufs["lse"]).abs().max() <= 2e-3


def test_serving_step_captured_and_replayed_as_the_cache_grows(bsa, pipe):
    """One graph of append + select + attend, replayed with new inputs and lengths in the same buffers, gives the
    eager step's bits; two graphs with workspaces of their own may run at once."""
    B, Hq, Hkv, d, nb, kb = 4, 16, 4, 128, 6, 2
    g = torch.Generator().manual_seed(13)
    sides = []
    for _ in range(2):
        pools = [t.cuda() for t in _pools(B * nb, Hkv, d, seed=1)]
        table = torch.arange(B * nb, dtype=torch.int32).view(B, nb).cuda()
        lens = torch.tensor([0, 62, 63, 190], dtype=torch.int32, device="cuda")
        start = torch.randn((B, Hkv, 256, d), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
        q = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda")
        step = pipe.QuantDecodeStep(q, *pools, table, torch.zeros_like(lens), kb=kb)
        step.append(start, start, new_lens=lens)
        step.seq_lens = lens
        k = torch.zeros((B, Hkv, 1, d), dtype=torch.bfloat16, device="cuda")
        sides.append((step, q, k, torch.zeros_like(k), lens))

    def turn(side):
        step, q, k, v, lens = side
        step.append(k, v)
        lens += 1
        step.run()
    eager, graphed = sides
    state = [t.clone() for t in (graphed[4], *[getattr(graphed[0], n) for n in ("k_pool", "v_pool", "k_exp", "v_exp")],
                                 graphed[0].bufs["kbar"])]
    side_stream = torch.cuda.Stream()
    side_stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side_stream):
        turn(graphed)
    torch.cuda.current_stream().wait_stream(side_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn(graphed)
    for dst, src in zip((graphed[4], *[getattr(graphed[0], n) for n in ("k_pool", "v_pool", "k_exp", "v_exp")],
                         graphed[0].bufs["kbar"]), state):
        dst.copy_(src)
    for t in range(70):
        for n, shape in ((1, (B, Hq, d)), (2, (B, Hkv, 1, d)), (3, (B, Hkv, 1, d))):
            x = torch.randn(shape, generator=g).bfloat16().cuda()
            eager[n].copy_(x)
            graphed[n].copy_(x)
        turn(eager)
        graph.replay()
        for name in ("o", "lse", "idx", "count"):
            assert torch.equal(eager[0].bufs[name], graphed[0].bufs[name]), (t, name)
    assert torch.equal(eager[0].k_pool, graphed[0].k_pool) and torch.equal(eager[0].bufs["kbar"], graphed[0].bufs["kbar"])


def test_calls_on_two_streams_at_once(bsa, pipe):
    """Two decodes and two backwards, each with its own workspace, on unordered streams, give what they give alone."""
    lens = [900, 300]
    steps, alone = [], []
    for seed in (0, 1):
        cache = _cache(lens, 2, 128, 15, seed=seed)
        q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        dev = [torch.from_numpy(x).cuda() for x in cache]
        dec = pipe.QuantDecodeStep(q, *dev, torch.tensor(lens, dtype=torch.int32).cuda())
        freq, _ = _rope_inputs(128, "half")
        enc = _encode_step(pipe, _qkv(1, 200, 8, 2, 128, torch.bfloat16, seed=seed).cuda(), 8, 2,
                           _weights(128, torch.bfloat16, True), freq, "half", None, 1.0)
        gen = torch.Generator().manual_seed(seed)
        grads = [torch.randn((1, h, 200, 128), generator=gen).cuda() for h in (8, 2, 2)]
        dec.run()
        enc.backward(*grads)
        alone.append([t.clone() for t in (dec.bufs["o"], dec.bufs["lse"], enc.bufs["d_qkv"], enc.bufs["d_q_weight"])])
        steps.append((dec, enc, grads))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for (dec, enc, grads), s in zip(steps, streams):
            dec.run(stream=s)
            enc.backward(*grads, stream=s)
    torch.cuda.synchronize()
    for (dec, enc, _), want in zip(steps, alone):
        for x, y in zip((dec.bufs["o"], dec.bufs["lse"], enc.bufs["d_qkv"], enc.bufs["d_q_weight"]), want):
            assert torch.equal(x, y)


def test_binding_refuses_wrong_types(bsa, pipe):
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((2, 2, 64, 128), dtype=torch.bfloat16, device="cuda")
    exps = torch.zeros((2, 2, 64), dtype=torch.uint8, device="cuda")
    codes = torch.zeros((2, 2, 64, 128), dtype=torch.float8_e4m3fn, device="cuda")
    table, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 2), (1,)))
    with pytest.raises(ValueError):
        pipe.QuantDecodeStep(q, pool, pool, exps, exps, table, lens).run()
    with pytest.raises(ValueError):
        pipe.QuantDecodeStep(q, codes, codes, exps, exps, table, lens.long()).run()
    with pytest.raises(ValueError):
        pipe.QuantDecodeStep(q, codes, codes, exps, exps.int(), table, lens).run()
    every = pipe.QuantDecodeStep(q, codes, codes.clone(), exps, exps.clone(), table, lens)
    with pytest.raises(ValueError):
        every.select()
    with pytest.raises(ValueError):
        every.attend(idx=torch.zeros((2, 2, 1), dtype=torch.int32, device="cuda"))
    k = torch.zeros((1, 2, 3, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        every.append(k, k, new_lens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        every.append(k.transpose(1, 2), k.transpose(1, 2))
    with pytest.raises(ValueError):
        every.append(k.float(), k.float())
    with pytest.raises(ValueError):
        every.read(k, k.clone(), starts=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        pipe.QkvStep(torch.zeros((1, 2, 4, 64), device="cuda"), 2, 1, q_weight=torch.ones(64).bfloat16().cuda(),
                     k_weight=torch.ones(64).cuda()).run()
    with pytest.raises(ValueError):
        bsa.bsa_topk_select_lens(torch.zeros((1, 4), device="cuda"), 1, 4, lens.long(), 1, 64, 1, table, 2)
