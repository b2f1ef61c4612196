"""The projections refuse to write over what they read: tiles of a row are read after others were written."""
import pytest
import torch

from lse_weighted_merge_dcp_amd import attn

pytestmark = pytest.mark.gpu


def test_out_over_the_inputs():
    g = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()       # noqa: E731
    o, w = rand(300, 4, 256), rand(4, 256, 256)
    before = o.clone(), w.clone()
    with pytest.raises(ValueError, match="lie over"):
        attn.latent_values(o, w, out=o)
    with pytest.raises(ValueError, match="lie over"):
        attn.latent_queries(o, w, out=o)
    with pytest.raises(ValueError, match="lie over"):
        attn.latent_values(o[:256], w, out=w.view(256, 4, 256))
    assert torch.equal(o, before[0]) and torch.equal(w, before[1])
    # beside them, and of nothing
    both = torch.zeros(300, 4, 512, dtype=torch.bfloat16, device="cuda")
    both[..., :256] = o
    assert torch.equal(attn.latent_values(both[..., :256], w, out=both[..., 256:]), attn.latent_values(o, w))
    attn.latent_values(o[:0], w, out=o[:0])
