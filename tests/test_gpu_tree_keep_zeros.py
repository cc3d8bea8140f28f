"""keep_kv8 with kept rows of zeros: they need no scale of their own, so the page that they go to may have one that is smaller
than their page's by any ratio that two scales can have."""
import pytest
import torch

import canvas_rope_rotary_amd as mr
import tree_ref as ref
from gpu_util import say
from test_gpu_kv8 import World, bits, i32
from test_gpu_tree import running

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32), (256, 16), (256, 64)])
@pytest.mark.parametrize("e", [17, 31, 32, 33, 119, 120])
def test_rows_of_zeros_from_a_large_scale(D, bs, e):
    """Zeros of either sign from a page of scale 2^e: to a new page (which goes to the least scale, 2^-96), to a page that holds
    rows under scales 2^126 to 2^129 times smaller, and beside rows of ordinary size.  Codes byte for byte."""
    say("keep zeros", D, bs, e)
    lens, past = [3 * bs] * 6, [bs, bs + 4, bs + 4, bs + 4, bs + 4, 0]
    w = World([a + b for a, b in zip(lens, past)], bs, 2, D, seed=D + bs + e)
    # position 2 bs + r is row r of the third page: of zeros under 2^e, in head 0 of K and head 1 of V
    for s in range(6):
        page, held = int(w.tables[s, 2]), int(w.tables[s, 1])
        w.kc.view(torch.uint8)[page, :8, 0], w.vc.view(torch.uint8)[page, :8, 1] = 0, 0
        w.kc.view(torch.uint8)[page, 1::2, 0, ::3] &= 0x80  # (rows past the eighth too: they are not kept)
        w.kc.view(torch.uint8)[page, 1, 0, 1::2] = 0x80
        w.vc.view(torch.uint8)[page, 2, 1] = 0x80
        w.ks[page, 0] = w.vs[page, 1] = 2.0 ** e
        if 1 <= s <= 4:
            w.ks[held, 0] = w.vs[held, 1] = 2.0 ** max(e - 125 - s, -96)
    first = bs - 4  # the token at position 2 bs of the sequences that begin at bs + 4
    lists = [[bs, bs + 1, bs + 2, bs + 7]] + [[first, first + 1, first + 2, first + 5]] * 3 + [[0, first + 1, first + 2, first + bs + 2],
                                                                                            [2 * bs + 1, 2 * bs + 2, 2 * bs + 3]]
    kept = [len(x) for x in lists]
    path = sum((x + [-1] * (n - len(x)) for x, n in zip(lists, lens)), [])
    caches = w.cache()
    mr.keep_kv8(i32(kept).cuda(), i32(path).cuda(), i32(running(lens)).cuda(), i32(past).cuda(), w.tables.cuda(), [tuple(caches)])
    ref.keep(kept, path, running(lens), past, w.tables.tolist(), w.kc, w.ks)
    ref.keep(kept, path, running(lens), past, w.tables.tolist(), w.vc, w.vs)
    assert torch.equal(caches[2].cpu(), w.ks) and torch.equal(caches[3].cpu(), w.vs)
    for got, want in zip(caches[:2], (w.kc, w.vc)):
        assert torch.equal(bits(got), want.view(torch.uint8))
