"""Which strided tensors have memory in common, against the sets of their bytes (CPU)."""

import random

import torch

from lm_head_cross_flce_amd import functional as F


def byte_set(t):
    n = t.element_size()
    at = [t.data_ptr()]
    for size, stride in zip(t.shape, t.stride()):
        at = [a + i * stride * n for a in at for i in range(size)]
    return {a + k for a in at for k in range(n)}


def test_against_the_bytes():
    rng = random.Random(1)
    buf = torch.zeros(400)
    half = buf.view(torch.bfloat16)
    hits = 0
    for _ in range(3000):
        views = []
        for _ in range(2):
            base = rng.choice((buf, half))
            shape = [rng.randint(1, 4) for _ in range(rng.randint(0, 3))]
            strides = [rng.choice((0, 1, 2, 3, 7, 12, 20, 60)) for _ in shape]
            span = sum((n - 1) * s for n, s in zip(shape, strides))
            views.append(base.as_strided(shape, strides, rng.randint(0, base.numel() - 1 - span)))
        want = bool(byte_set(views[0]) & byte_set(views[1]))
        hits += want
        assert F._share_memory(*views) == want, [(v.shape, v.stride(), v.storage_offset(), v.dtype) for v in views]
    assert hits > 50   # both answers occur


def test_views_of_one_buffer():
    buf = torch.zeros(3000, 2000)
    assert not F._share_memory(buf[:, ::2], buf[:, 1::2])
    assert not F._share_memory(buf[:, :700], buf[:, 700:])
    assert not F._share_memory(buf[::2], buf[1::2, 5:90])
    assert F._share_memory(buf[:, ::2], buf[:, ::2])
    assert F._share_memory(buf[:, :701], buf[:, 700:])
    assert F._share_memory(buf.T, buf[2999:, 1999:])
    assert not F._share_memory(buf[:0], buf)


def test_what_clipping_would_write_twice():
    buf = torch.zeros(40, 60)
    F._check_written([buf[:, ::2], buf[:, 1::2], torch.zeros(5)])
    F._check_written([buf[:, 20 * i:20 * i + 20] for i in range(3)])
    for bad in ([buf[:, ::2], buf[:, ::2]], [buf[:, :31], torch.zeros(3), buf[:, 30:]], [buf, buf[:, 3]]):
        try:
            F._check_written(bad)
        except ValueError:
            continue
        raise AssertionError(bad)
