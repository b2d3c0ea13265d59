"""Host side of the step objects of the norm + rotation and the quantised
cache: fields replaced by others of the wrong size, and buffers that the
caller brings and that are too small, are refused before anything reaches the
library.  No device is touched."""
import pytest
import torch

import top_block_sparse_bsa_b200 as bsa  # noqa: F401
from top_block_sparse_bsa_b200 import pipeline

BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def _encode(**kw):
    a = dict(qkv=torch.zeros((2, 3, 8, 64), dtype=BF16), Hq=4, Hkv=2, q_weight=torch.ones(64, dtype=BF16),
             k_weight=torch.ones(64, dtype=BF16), positions=torch.zeros((2, 3), dtype=I32))
    a.update(kw)
    return pipeline.QkvStep(a.pop("qkv"), a.pop("Hq"), a.pop("Hkv"), **a)


@pytest.mark.parametrize("field,value", [
    ("qkv", torch.zeros((2, 4, 8, 64), dtype=BF16)), ("qkv", torch.zeros((2, 3, 8, 32), dtype=BF16)),
    ("positions", torch.zeros((2, 2), dtype=I32)), ("positions", torch.zeros(6, dtype=I32)),
    ("q_weight", torch.ones(32, dtype=BF16)), ("k_weight", torch.ones((1, 64), dtype=BF16)), ("Hq", 2), ("Hkv", 4),
    ("bufs", {"k": torch.zeros((2, 2, 2, 64), dtype=BF16)})])
def test_encode_step_refuses_replaced_fields_of_another_size(field, value):
    step = _encode()
    setattr(step, field, value)
    grads = [torch.zeros((2, h, 3, 64)) for h in (4, 2, 2)]
    for _ in range(2):                       # and goes on refusing
        with pytest.raises(ValueError):
            step.run()
        with pytest.raises(ValueError):
            step.backward(*grads)


def test_encode_step_refuses_small_buffers():
    for name in ("q", "k", "v"):
        with pytest.raises(ValueError):
            _encode(bufs={name: torch.zeros((2, 2, 2, 64), dtype=BF16)})
    for name in ("d_q_weight", "d_k_weight"):
        step = _encode(bufs={name: torch.zeros(32)})
        with pytest.raises(ValueError):
            step.backward(*[torch.zeros((2, h, 3, 64)) for h in (4, 2, 2)])


def _decode(kb=2, **kw):
    pool = torch.zeros((9, 2, 64, 64), dtype=U8)
    return pipeline.QuantDecodeStep(torch.zeros((3, 4, 64), dtype=BF16), pool, pool.clone(), pool[..., 0].contiguous(),
                                    pool[..., 0].contiguous(), torch.zeros((3, 5), dtype=I32),
                                    torch.zeros(3, dtype=I32), kb=kb, **kw)


# a table of more blocks, among others: the summary that appends write is laid out by the table's width
@pytest.mark.parametrize("field,value", [
    ("q", torch.zeros((2, 4, 64), dtype=BF16)), ("q", torch.zeros((3, 2, 64), dtype=BF16)),
    ("k_pool", torch.zeros((9, 1, 64, 64), dtype=U8)), ("k_pool", torch.zeros((9, 2, 64, 32), dtype=U8)),
    ("block_table", torch.zeros((3, 8), dtype=I32)), ("block_table", torch.zeros((2, 5), dtype=I32)),
    ("seq_lens", torch.zeros(2, dtype=I32)), ("kb", 3), ("kb", None),
    ("bufs", {"kbar": torch.zeros((3, 2, 4, 64))})])
def test_decode_step_refuses_replaced_fields_of_another_size(field, value):
    step = _decode()
    setattr(step, field, value)
    x = torch.zeros((3, 2, 1, 64), dtype=BF16)
    for call in (step.run, step.select, step.attend, lambda: step.append(x, x), lambda: step.read(x, x), step.run):
        with pytest.raises(ValueError):
            call()


def test_decode_step_refuses_small_buffers_and_a_late_kb():
    for name, shape in (("kbar", (3, 2, 4, 64)), ("qbar", (3, 1, 64)), ("scores", (3, 2, 4)), ("idx", (3, 2, 2)),
                        ("count", (3,)), ("o", (3, 2, 64)), ("lse", (3, 3))):
        with pytest.raises(ValueError):
            _decode(bufs={name: torch.zeros(shape)})
    step = _decode(kb=None)
    step.kb = 2
    with pytest.raises(ValueError):
        step.select()


def test_encode_step_refuses_small_gradient_buffers_that_come_with_a_workspace():
    for small in ("d_q_weight", "d_k_weight"):
        bufs = {"d_q_weight": torch.zeros(64), "d_k_weight": torch.zeros(64), "qkv_workspace": torch.zeros(1024, dtype=U8)}
        bufs[small] = torch.zeros(32)
        step = _encode(bufs=bufs)
        with pytest.raises(ValueError):
            step.backward(*[torch.zeros((2, h, 3, 64)) for h in (4, 2, 2)])
