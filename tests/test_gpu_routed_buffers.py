"""GPU: the holders of experts, adapters and row groups reference tensors.
A tensor that is put in another's place, or whose storage is replaced (as a
module's conversion does), is what the next call reads."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev
from routed_util import Experts, device_groups

pytestmark = pytest.mark.gpu

N, K, R, COUNT, ROWS = 40, 128, 8, 3, 12


def inputs():
    import torch
    rng = np.random.default_rng(0)
    f = lambda *s: to_dev(rng.standard_normal(s).astype(np.float32))
    h = lambda *s: f(*s).half()
    ids = rng.integers(0, COUNT, ROWS).astype(np.int32)
    return f, h, ids


def test_adapters():
    import torch
    f, h, ids = inputs()
    g, *_ = device_groups(ids, COUNT)
    x, base = h(ROWS, K), f(ROWS, N)
    old = h(COUNT, R, K), h(COUNT, N, R), f(COUNT)  # held, so that nothing of theirs is freed
    ad = qw.Adapters(*old)
    qw.qw_lora_add(ad, x, g, base)
    new = h(COUNT, R, K), h(COUNT, N, R), f(COUNT)
    now = list(old)
    for i, name in enumerate(("A", "B", "scale")):
        setattr(ad, name, new[i])
        now[i] = new[i]
        assert torch.equal(qw.qw_lora_add(ad, x, g, base), qw.qw_lora_add(qw.Adapters(*now), x, g, base)), name
    p = torch.nn.Parameter(old[0].clone(), requires_grad=False)
    ad = qw.Adapters(p, old[1], old[2])
    held = p.data
    p.data = new[0].clone()
    want = qw.qw_lora_add(qw.Adapters(new[0], old[1], old[2]), x, g, base)
    assert torch.equal(qw.qw_lora_add(ad, x, g, base), want)
    del held


def test_experts():
    import torch
    f, h, ids = inputs()
    g, *_ = device_groups(ids, COUNT)
    x = h(ROWS, K)
    for fmt, n_out in (("2bit", 5), ("int4", 5), ("nf4", 0)):
        a, b = Experts(fmt, COUNT, N, K, n_out, seed=1), Experts(fmt, COUNT, N, K, n_out, seed=2)
        want = qw.qgemm_experts(b.ew, x, g)
        held = []
        for name in ("codes", "scales", "out_idx", "out_w", "out_mask"):
            held.append(getattr(a.ew, name))
            setattr(a.ew, name, getattr(b.ew, name))
        assert torch.equal(qw.qgemm_experts(a.ew, x, g), want), fmt


def test_groups():
    import torch
    f, h, ids = inputs()
    ex = Experts("nf4", COUNT, N, K, 0, seed=1)
    x = h(ROWS, K)
    a, *_ = device_groups(ids, COUNT)
    b, *_ = device_groups(ids[::-1].copy(), COUNT)
    held = a.offsets, a.rows
    a.offsets, a.rows = b.offsets, b.rows
    assert torch.equal(qw.qgemm_experts(ex.ew, x, a), qw.qgemm_experts(ex.ew, x, b))
    del held


def test_buffers_that_do_not_fit_are_refused():
    """What the constructors refuse is refused after a replacement too."""
    import torch
    f, h, ids = inputs()
    g, *_ = device_groups(ids, COUNT)
    x, base = h(ROWS, K), f(ROWS, N)
    ad = qw.Adapters(h(COUNT, R, K), h(COUNT, N, R), f(COUNT))
    keep = ad.A, ad.B, ad.scale
    for name, t in (("A", h(COUNT, R + 8, K)), ("B", h(COUNT, N, R)[:, ::2]), ("scale", f(COUNT + 1)), ("A", f(COUNT, R, K)),
                    ("scale", torch.ones(COUNT))):
        was = getattr(ad, name)
        setattr(ad, name, t)
        with pytest.raises((TypeError, ValueError)):
            qw.qw_lora_add(ad, x, g, base)
        setattr(ad, name, was)
    qw.qw_lora_add(ad, x, g, base)
    ex = Experts("nf4", COUNT, N, K, 0, seed=1)
    was = ex.ew.codes
    ex.ew.codes = was[:-16]
    with pytest.raises(ValueError):
        qw.qgemm_experts(ex.ew, x, g)
    ex.ew.codes = was
    offs = g.offsets
    g.offsets = offs[:-1]
    with pytest.raises(ValueError):
        qw.qgemm_experts(ex.ew, x, g)
    g.offsets, g.rows = offs, g.rows.long()
    with pytest.raises(TypeError):
        qw.qgemm_experts(ex.ew, x, g)
    del keep


def test_a_refused_buffer_leaves_the_holder_as_it_was():
    import torch
    f, h, ids = inputs()
    g, *_ = device_groups(ids, COUNT)
    x, base = h(ROWS, K), f(ROWS, N)
    ad = qw.Adapters(h(COUNT, R, K), h(COUNT, N, R), f(COUNT))
    want = qw.qw_lora_add(ad, x, g, base)
    was = ad.A, ad.B, ad.scale
    for bad in ((h(COUNT + 1, R, K + 8), was[1], was[2]), (was[0], h(COUNT, N + 8, R + 8), was[2]), (was[0], was[1], f(COUNT - 1))):
        ad.A, ad.B, ad.scale = bad
        with pytest.raises(ValueError):
            qw.qw_lora_add(ad, x, g, base)
        ad.A, ad.B, ad.scale = was
        assert torch.equal(qw.qw_lora_add(ad, x, g, base), want)
    # adapters of another rank and number are taken as a whole
    ad.A, ad.B, ad.scale = h(COUNT + 2, 2 * R, K), h(COUNT + 2, N, 2 * R), f(COUNT + 2)
    g, *_ = device_groups(ids, COUNT + 2)
    assert torch.equal(qw.qw_lora_add(ad, x, g, base), qw.qw_lora_add(qw.Adapters(ad.A, ad.B, ad.scale), x, g, base))
