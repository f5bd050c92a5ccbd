"""Rotary positions between parts of one tensor: what shares no element is turned, and the rest of the tensor stays; what does is
refused before anything is written."""
import pytest
import torch

from topology_construction_amd import binding

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


APART = {
    "queries into keys": (lambda t: t[:, :4], lambda t: t[:, 4:8]),
    "values into queries": (lambda t: t[:, 8:], lambda t: t[:, :4]),
    "every other head": (lambda t: t[:, 0:8:2], lambda t: t[:, 1:8:2]),
    "every other row": (lambda t: t[0:60:2, :4], lambda t: t[1:60:2, :4]),
    "every other row into rows": (lambda t: t[0:60:2, :4], lambda t: t[:30, 4:8]),
    "one row for all": (lambda t: t[:1, :4].expand(60, 4, 40), lambda t: t[:, 4:8]),
    "one head for all": (lambda t: t[:, :1].expand(60, 4, 40), lambda t: t[:, 1:5]),
    "parts of a head": (lambda t: t[..., :20], lambda t: t[..., 20:]),
    "heads before rows": (lambda t: t[:4].transpose(0, 1), lambda t: t[4:8].transpose(0, 1)),
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("form", APART)
def test_parts_that_share_nothing(form, interleaved, dtype):
    t = torch.randn(60, 12, 40, generator=_gen(1), device="cuda").to(dtype)
    x, out = (part(t) for part in APART[form])
    pairs = min(7, x.shape[2] // 2)
    pos = torch.randint(-99, 99, (x.shape[0], 1), generator=_gen(2), device="cuda", dtype=torch.int32)
    freqs = torch.rand(pairs, generator=_gen(3), device="cuda")
    want = t.clone()
    APART[form][1](want).copy_(binding.tc_rotary(x.clone(), pos, freqs, interleaved=interleaved))
    assert binding.tc_rotary(x, pos, freqs, interleaved=interleaved, out=out) is out
    assert torch.equal(t, want)


SHARED = {
    "heads": (lambda t: t[:, :3], lambda t: t[:, 2:5]),
    "heads, before": (lambda t: t[:, 1:4], lambda t: t[:, 0:3]),
    "rows": (lambda t: t[:50, :3], lambda t: t[1:51, :3]),
    "channels": (lambda t: t[..., :20], lambda t: t[..., 19:39]),
    "every other head": (lambda t: t[:, 0:8:2], lambda t: t[:, 2:10:2]),
    "into the one row": (lambda t: t[5:6, :4].expand(60, 4, 40), lambda t: t[:, 2:6]),
    "other strides": (lambda t: t[0:60:2, :4], lambda t: t[:30, 3:7]),
    "itself, turned": (lambda t: t[:12, :12], lambda t: t[:12, :12].transpose(0, 1)),
}


@pytest.mark.parametrize("form", SHARED)
def test_parts_that_overlap_are_refused(form):
    t = torch.randn(60, 12, 40, generator=_gen(1), device="cuda")
    before = t.clone()
    x, out = (part(t) for part in SHARED[form])
    pos = torch.zeros(x.shape[0], 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        binding.tc_rotary(x, pos, torch.ones(7, device="cuda"), out=out)
    assert torch.equal(t, before)


def test_itself_in_other_words():
    """The same place is x, whatever the strides of what there is one of."""
    t = torch.randn(60, 12, 40, generator=_gen(1), device="cuda")
    pos, freqs = torch.arange(60, dtype=torch.int32, device="cuda")[:, None], torch.rand(9, generator=_gen(3), device="cuda")
    want = binding.tc_rotary(t[:, :1].clone(), pos, freqs)
    x = t[:, :1]
    binding.tc_rotary(x, pos, freqs, out=torch.as_strided(t, (60, 1, 40), (480, 7, 1)))
    assert torch.equal(x, want)
    want = binding.tc_rotary(t[3:4].clone(), pos[:1], freqs)
    binding.tc_rotary(t[3:4], pos[:1], freqs, out=torch.as_strided(t, (1, 12, 40), (1, 40, 1), 3 * 480))
    assert torch.equal(t[3:4], want)
