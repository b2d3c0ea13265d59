"""GPU tests at the edges of the norm + rotation, the quantised cache and the
decode over it: rows that only pad a block's work, fields of a step that
change between calls, magnitudes at the ends of the types, and equal bits on
every run.

Tolerances count roundings.  Half a step of a type is finfo(t).eps / 2
relative to the value: bf16 2^-8, fp32 2^-24.
"""
import math

import numpy as np
import pytest
import torch

import plain_operators as plain
from test_gpu_operators import HALF, _cache, _check_decode, _cuda, _encode_step, _qkv, _rope_inputs, _weights

pytestmark = pytest.mark.gpu


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


# ------------------------------------------------------------ norm + rotation

# N = 2500: enough tokens for full runs of heads (4 rows of bf16 or 2 of fp32 in flight), whose last one is partial
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [1, 21, 2500])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (4, 2, 128), (5, 3, 64), (7, 1, 128), (8, 4, 64)])
def test_weights_gradients_without_eps(pipe, Hq, Hkv, d, N, dtype):
    """eps = 0: a head run's padding, whose mean of squares is 0, must not reach the weights' gradients."""
    qkv = _qkv(1, N, Hq, Hkv, d, dtype, spread=0.5)
    w = _weights(d, dtype, True)
    freq, _ = _rope_inputs(d, "half")
    g = torch.Generator().manual_seed(4)
    grads = [torch.randn((1, h, N, d), generator=g) for h in (Hq, Hkv, Hkv)]
    step = _encode_step(pipe, qkv.cuda(), Hq, Hkv, w, freq, "half", None, 1.0, eps=0.0)
    got = step.backward(*(x.cuda() for x in grads))
    want, (size, dw_size) = plain.encode_grad(qkv.double(), Hq, Hkv, w[0].double(), w[1].double(), 0.0, freq, "half",
                                              None, 1.0, *(x.double() for x in grads))
    err = (got["d_qkv"].cpu().double() - want[0]).abs()
    # as with eps: two sums of d products, about 30 roundings on the longest way
    assert bool((err <= HALF[dtype] * want[0].abs() + 2.0 ** -18 * size).all()), (err / (size + 1e-30)).max()
    rows = N * max(Hq, Hkv)
    for name, x, s in zip(("d_q_weight", "d_k_weight"), want[1:], dw_size):
        # at most `rows` terms on one lane's way, each 2^-20 off, then 32 groups
        err = (got[name].cpu().double() - x).abs()
        assert bool((err <= ((rows + 32) * 2.0 ** -24 + 2.0 ** -20) * s).all()), name


@pytest.mark.parametrize("change", ["inv_freq", "a shorter inv_freq", "layout", "rope_scale", "no rotation", "all"])
def test_replaced_rotation_counts_from_the_next_call_on(pipe, change):
    """A step whose frequencies, layout or scale are replaced gives, forward and backward, what a new step gives."""
    Hq, Hkv, N, d = 4, 2, 40, 128
    qkv = _qkv(1, N, Hq, Hkv, d, torch.bfloat16, spread=0.5).cuda()
    w = _weights(d, torch.bfloat16, True)
    freq, _ = _rope_inputs(d, "half")
    g = torch.Generator().manual_seed(4)
    grads = [torch.randn((1, h, N, d), generator=g).cuda() for h in (Hq, Hkv, Hkv)]
    new = {"inv_freq": dict(inv_freq=freq / 4), "a shorter inv_freq": dict(inv_freq=freq[:24].clone()),
           "layout": dict(layout=2), "rope_scale": dict(rope_scale=0.5), "no rotation": dict(inv_freq=None),
           "all": dict(inv_freq=freq[:32] / 3, layout=2, rope_scale=1.5)}[change]
    step = _encode_step(pipe, qkv, Hq, Hkv, w, freq, "half", None, 1.0)
    first = step.run()["q"].clone()
    step.backward(*grads)
    for name, value in new.items():
        setattr(step, name, _cuda(value) if name == "inv_freq" else value)
    names = ("q", "k", "v", "d_qkv", "d_q_weight", "d_k_weight")
    got = {**step.run(), **step.backward(*grads)}
    f, layout, scale = new.get("inv_freq", freq), new.get("layout", 1), new.get("rope_scale", 1.0)
    fresh = _encode_step(pipe, qkv, Hq, Hkv, w, f, ("none", "half", "pairs")[layout], None, scale)
    want = {**fresh.run(), **fresh.backward(*grads)}
    assert all(torch.equal(got[n], want[n]) for n in names)
    assert not torch.equal(got["q"], first)
    # and back, to a step that was built without a rotation too
    step.inv_freq, step.layout, step.rope_scale = freq.cuda(), 1, 1.0
    assert torch.equal(step.run()["q"], first)
    bare = _encode_step(pipe, qkv, Hq, Hkv, w, None, "half", None, 1.0)
    bare.run()
    bare.inv_freq = freq.cuda()
    assert torch.equal(bare.run()["q"], first)


def test_frequencies_are_checked_like_every_tensor(bsa, pipe):
    qkv = _qkv(1, 5, 2, 1, 64, torch.bfloat16).cuda()
    freq, _ = _rope_inputs(64, "half")
    step = _encode_step(pipe, qkv, 2, 1, (None, None), freq, "half", None, 1.0)
    for bad in (freq, freq.float().cuda(), torch.stack([freq, freq], 1)[:, 0].cuda()[::2]):
        step.inv_freq = bad
        with pytest.raises(ValueError):
            step.run()
        with pytest.raises(ValueError):
            step.backward(*(torch.zeros((1, h, 5, 64), device="cuda") for h in (2, 1, 1)))

    class Elsewhere:                     # a tensor of another device
        dtype, device, is_cuda = torch.float64, "cuda:99", True

        def get_device(self):
            return 99

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 256
    rope = bsa.make_rope(bsa.BSA_ROPE_HALF, freq.cuda())
    rope.freq = Elsewhere()
    b = step.bufs
    with pytest.raises(ValueError):
        bsa.bsa_qkv_norm_rope(step.shape, qkv, None, None, 0.0, rope, None, b["q"], b["k"], b["v"])
    # the frequencies live as long as the rotation made of them
    rope = bsa.make_rope(bsa.BSA_ROPE_HALF, (freq / 2).cuda())
    torch.full((32,), 7.0, dtype=torch.float64, device="cuda")
    bsa.bsa_qkv_norm_rope(step.shape, qkv, None, None, 0.0, rope, None, b["q"], b["k"], b["v"])
    want = _encode_step(pipe, qkv, 2, 1, (None, None), freq / 2, "half", None, 1.0).run()
    assert torch.equal(b["q"], want["q"])


def test_replaced_tensors_of_the_same_size_count_from_the_next_call_on(pipe):
    Hq, Hkv, N, d = 4, 2, 40, 128
    freq, _ = _rope_inputs(d, "half")
    g = torch.Generator().manual_seed(4)
    grads = [torch.randn((2, h, N, d), generator=g).cuda() for h in (Hq, Hkv, Hkv)]
    pos = [torch.randint(0, 5000, (2, N), generator=g).int() for _ in range(2)]
    qkv = [_qkv(2, N, Hq, Hkv, d, torch.bfloat16, seed=s, spread=0.5).cuda() for s in (0, 1)]
    w = [_weights(d, torch.bfloat16, True, seed=s) for s in (5, 6)]
    step = _encode_step(pipe, qkv[0], Hq, Hkv, w[0], freq, "half", pos[0], 1.0)
    step.run()
    step.backward(*grads)
    step.qkv, step.positions, step.q_weight, step.k_weight = qkv[1], pos[1].cuda(), w[1][0].cuda(), w[1][1].cuda()
    got = {**step.run(), **step.backward(*grads)}
    fresh = _encode_step(pipe, qkv[1], Hq, Hkv, w[1], freq, "half", pos[1], 1.0)
    want = {**fresh.run(), **fresh.backward(*grads)}
    assert all(torch.equal(got[n], want[n]) for n in ("q", "k", "v", "d_qkv", "d_q_weight", "d_k_weight"))
    step.q_weight = step.k_weight = None                     # without norms, gradients of no weights
    fresh = _encode_step(pipe, qkv[1], Hq, Hkv, (None, None), freq, "half", pos[1], 1.0)
    assert torch.equal(step.backward(*grads)["d_qkv"], fresh.backward(*grads)["d_qkv"])


@pytest.mark.parametrize("handle", [False, True])
def test_gradients_made_on_another_stream_take_no_memory_that_this_one_still_reads(pipe, handle):
    """The first backward takes memory for its outputs; on another stream it must not be what this stream has given back
    and its queued work is still to read."""
    qkv = _qkv(1, 512, 6, 1, 128, torch.bfloat16, spread=0.3).cuda()
    step = _encode_step(pipe, qkv, 6, 1, (None, None), None, "half", None, 1.0)
    grads = [torch.ones((1, h, 512, 128), device="cuda") for h in (6, 1, 1)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    x = torch.full_like(qkv, 7.0)
    torch.cuda._sleep(50_000_000)                            # some 30 ms
    y = x + 0
    del x
    step.backward(*grads, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert bool((y == 7).all())
    assert bool((step.bufs["d_qkv"] == 1).all())


def test_encode_and_backward_past_32_bits(pipe):
    """More than 2^31 channels: the last tokens come out as in a call of their own."""
    Hq, Hkv, N, d, tail = 32, 8, 360_000, 128, 70
    freq, _ = _rope_inputs(d, "half")
    w = _weights(d, torch.bfloat16, True)
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((1, N, Hq + 2 * Hkv, d), generator=g, device="cuda", dtype=torch.bfloat16)
    assert qkv.numel() > 2 ** 31
    pos = torch.arange(N, dtype=torch.int32).view(1, N)
    step = _encode_step(pipe, qkv, Hq, Hkv, w, freq, "half", pos, 1.0)
    last = _encode_step(pipe, qkv[:, -tail:].contiguous(), Hq, Hkv, w, freq, "half", pos[:, -tail:].contiguous(), 1.0)
    got, want = step.run(), last.run()
    assert all(torch.equal(got[n][:, :, -tail:], want[n]) for n in "qkv")
    grads = [torch.zeros((1, h, N, d), device="cuda") for h in (Hq, Hkv, Hkv)]      # none but the last tokens'
    for x in grads:
        x[:, :, -tail:] = torch.randn((1, x.shape[1], tail, d), generator=g, device="cuda")
    got, want = step.backward(*grads), last.backward(*(x[:, :, -tail:].contiguous() for x in grads))
    assert torch.equal(got["d_qkv"][:, -tail:], want["d_qkv"]) and not got["d_qkv"][:, :-tail].any()
    for name in ("d_q_weight", "d_k_weight"):
        # the same terms, at most tail * Hq, in sums of another order
        assert bool(((got[name] - want[name]).abs() <= tail * Hq * 2.0 ** -24 * 2 * want[name].abs().max()).all())


@pytest.mark.parametrize("brought", [(), ("qkv_workspace",), ("d_q_weight",), ("d_k_weight", "qkv_workspace"), ("d_qkv",)])
def test_backward_makes_the_buffers_that_the_caller_did_not_bring(pipe, brought):
    qkv = _qkv(1, 70, 3, 1, 64, torch.bfloat16, spread=0.5).cuda()
    w = _weights(64, torch.bfloat16, True)
    freq, _ = _rope_inputs(64, "half")
    grads = [torch.randn((1, h, 70, 64), generator=torch.Generator().manual_seed(h)).cuda() for h in (3, 1, 1)]
    want = _encode_step(pipe, qkv, 3, 1, w, freq, "half", None, 1.0).backward(*grads)
    bufs = {n: torch.empty_like(want[n]) for n in brought}
    step = pipe.QkvStep(qkv, 3, 1, q_weight=w[0].cuda(), k_weight=w[1].cuda(), eps=1e-5, inv_freq=freq.cuda(),
                        bufs=dict(bufs))
    got = step.backward(*grads)
    assert all(torch.equal(got[n], want[n]) for n in ("d_qkv", "d_q_weight", "d_k_weight"))
    assert all(got[n] is bufs[n] for n in brought)


# --------------------------------------------------------------------- decode

@pytest.mark.parametrize("Hq,d", [(4, 128), (16, 64)])
@pytest.mark.parametrize("exponent,up", [(236, -117), (244, -124), (10, 100), (10, 115), (120, -100)])
def test_decode_of_keys_and_queries_at_opposite_ends(bsa, exponent, up, Hq, d):
    """Keys and queries near the two ends of fp32 with logits of ordinary size: no partial product leaves fp32."""
    lens = [500, 33]
    cache = _cache(lens, 1, d, 9, seed=3)
    ke = np.where(cache[2] == 255, 255, np.clip(cache[2].astype(int) - 117 + exponent, 10, 246)).astype(np.uint8)
    q = (2.0 ** up * torch.randn((2, Hq, d), generator=torch.Generator().manual_seed(6))).bfloat16()
    # Some logits lie 100 apart here.  A weight is rounded to fp16 with the largest y = logit + value exponent of its
    # warp's keys at 2^8 or above (the reference is a y, and no y passes it by more than 7 octaves at 2^15): an error of
    # at most half of fp16's least step, 2^-25, is 2^-33 of the largest weight, times a code of at most 448, for each of
    # at most 500 keys; the largest weight itself is at most 1 in units of the largest value exponent's power of two.
    least = 500 * 2.0 ** -33 * 448 * 2.0 ** (int(cache[3][cache[3] != 255].max()) - 127)
    _check_decode(bsa, q, (cache[0], cache[1], ke, cache[3], cache[4]), lens, None, least=least)


def _decode_step(pipe, seed, lens, kb, **kw):
    cache = _cache(lens, 2, 128, 12, seed=seed)
    q = torch.randn((len(lens), 8, 128), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    step = pipe.QuantDecodeStep(q, *(torch.from_numpy(x).cuda() for x in cache),
                                torch.tensor(lens, dtype=torch.int32).cuda(), kb=kb, **kw)
    if kb is not None:
        step.bufs["kbar"].copy_(torch.randn(step.bufs["kbar"].shape, generator=torch.Generator().manual_seed(seed)))
    return step


def test_replaced_decode_tensors_of_the_same_size_count_from_the_next_call_on(pipe):
    a, b = _decode_step(pipe, 1, [700, 40, 333], 3), _decode_step(pipe, 2, [64, 768, 0], 2)
    want = {n: b.run()[n].clone() for n in ("o", "lse", "count")}
    a.run()
    for name in ("q", "k_pool", "v_pool", "k_exp", "v_exp", "block_table", "seq_lens"):
        setattr(a, name, getattr(b, name))
    a.kb = 2                                                 # fewer than it was built for: the lists end earlier
    a.bufs["kbar"].copy_(b.bufs["kbar"])
    got = a.run()
    assert torch.equal(got["idx"][..., :3], b.bufs["idx"]) and bool((got["idx"][..., 3:] == -1).all())
    # the lists' lengths decide where rows are cut, and so in which order a row's keys are summed: an output may fall on
    # the other side of a rounding
    assert torch.equal(got["count"], want["count"])
    assert torch.allclose(got["o"].float(), want["o"].float(), rtol=2.0 ** -7, atol=2.0 ** -9)
    assert torch.allclose(got["lse"], want["lse"], rtol=2.0 ** -18)


def test_a_step_of_every_block_attends_every_block_with_another_step_s_buffers(pipe):
    lens = [700, 40, 333]
    kept = _decode_step(pipe, 1, lens, 3)
    alone = _decode_step(pipe, 1, lens, None).run()["o"].clone()
    workspace = torch.empty_like(_decode_step(pipe, 1, lens, None).bufs["workspace"])
    every = _decode_step(pipe, 1, lens, None, bufs={**kept.bufs, "workspace": workspace})
    few = kept.run()["o"].clone()
    assert torch.equal(every.run()["o"], alone) and not torch.equal(few, alone)
