"""What the calls for trees of drafted tokens refuse to write, through the binding: memory that they would write twice, or read
and write at once."""
import pytest
import torch

import canvas_rope_rotary_amd as mr
from test_gpu_kv8 import World, bits, i32

pytestmark = pytest.mark.gpu


def test_keep_refuses_a_cache_twice():
    """The same cache for two layers, K in V's place, a layer that begins within another: refused, and nothing is moved."""
    w = World([60], 16, 2, 128, seed=81)
    kc, vc, ks, vs = w.cache()
    k2, v2, ks2, vs2 = w.cache()
    args = (i32([3]).cuda(), i32([0, 2, 4, -1, -1, -1]).cuda(), i32([0, 6]).cuda(), i32([40]).cuda(), w.tables.cuda())
    wide = torch.zeros(w.nb + 1, *kc.shape[1:], dtype=torch.uint8, device="cuda")
    for caches in ([(kc, vc, ks, vs)] * 2, [(kc, kc, ks, vs)], [(kc, vc, ks, ks)], [(kc, vc, ks, vs), (k2, vc, ks2, vs2)],
                   [(kc, vc, ks, vs), (k2, v2, ks2, vs)], [(wide[1:], wide[:-1], ks, vs)]):
        with pytest.raises(mr.MropeError, match="share"):
            mr.keep_kv8(*args, caches)
    assert torch.equal(bits(kc), bits(w.kc)) and torch.equal(bits(vc), bits(w.vc)) and torch.equal(ks.cpu(), w.ks)
    mr.keep_kv8(*args, [(kc, vc, ks, vs), (k2, v2, ks2, vs2)])
    assert torch.equal(bits(kc), bits(k2)) and torch.equal(bits(vc), bits(v2)) and not torch.equal(bits(kc), bits(w.kc))
