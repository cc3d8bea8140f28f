"""attend_tree_kv8 over chunks of contexts: as long as a workgroup looks its pages up more than once, and results that repeat."""
import random

import pytest
import torch

import canvas_rope_rotary_amd as mr
import tree_ref as ref
from gpu_util import say
from test_gpu_kv8 import World, i32
from test_gpu_kv8_precision import within
from test_gpu_tree import running, tree_masks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_narrow_chunks_of_64_dims_past_a_look_up(dtype):
    """Eight waves look pages up anew after 8,192 tokens of a chunk.  Three trees in 64 KV heads of 64 dims are tiles of 32 rows, and
    512 workgroups that run at once leave 8 chunks a head, so contexts of 27,000 positions are cut in two or three: chunks of 9,000 to
    14,000."""
    say("tree look-ups", dtype)
    w = World([640], 16, 64, 64, seed=180)
    lens, ctx = [2, 1, 2], [27000, 26991, 27300]
    w.tables = w.tables[:, :40].repeat(3, 43)[:, :1707]
    w.tables[1] = w.tables[1].flip(0)
    mask = tree_masks(lens, 1, random.Random(3), "tree")
    cu, q = running(lens), w.heads(sum(lens), 64, dtype)
    out, lse = mr.attend_tree_kv8(q.cuda(), i32(cu).cuda(), i32(ctx).cuda(), mask.cuda(), w.tables.cuda(), *w.cache(), return_lse=True)
    heads = [0, 63]
    part = [x[:, :, heads] for x in (w.kc, w.vc)] + [x[:, heads] for x in (w.ks, w.vs)]
    o, z, spread, amp = ref.attend_tree(q[:, heads], cu, ctx, mask.tolist(), w.tables.tolist(), *part)
    within(out[:, heads].cpu().double(), lse[:, heads].cpu().double(), o, z, spread, amp, dtype, 64, 27300, "look-ups")


@pytest.mark.parametrize("dtype,D,hq,hk,n", [("bf16", 256, 8, 2, 16), ("f16", 128, 16, 4, 9), ("bf16", 64, 4, 4, 40), ("f32", 256, 8, 2, 8)])
def test_results_repeat(dtype, D, hq, hk, n):
    """Long contexts in chunks that are joined: the same bits from call to call, whatever the output and workspace held, with other
    calls in between and on two streams at once; and from tensors that another call's inputs are copied into."""
    say("tree repeats", dtype, D)
    worlds = []
    for seed in (181, 182):
        w = World([5000 + n, 61 + n, 3000 + n], 64, hk, D, seed=seed)
        mask = tree_masks([n] * 3, 1, random.Random(seed), "tree")
        worlds.append([w.heads(3 * n, hq, dtype).cuda(), mask.cuda(), w.tables.cuda(), *w.cache()])
    cu, ctx = i32([0, n, 2 * n, 3 * n]).cuda(), i32([5000 + n, 61 + n, 3000 + n]).cuda()

    def call(x, **kw):
        return mr.attend_tree_kv8(x[0], cu, ctx, *x[1:], return_lse=True, **kw)

    want = [call(x) for x in worlds]
    need = mr.attend_tree_kv8_workspace_bytes(worlds[0][0], 3, worlds[0][2], worlds[0][3])
    assert need > 0
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    for turn in range(20):
        x, (o, z) = worlds[turn % 2], want[turn % 2]
        got = call(x, workspace=ws, out=torch.full_like(o, float("nan"))) if turn % 4 < 2 else call(x)
        assert torch.equal(got[0], o) and torch.equal(got[1], z), turn
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for turn in range(10):
        got = []
        for s, x in zip(streams, worlds):
            with torch.cuda.stream(s):
                got.append(call(x))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, v in zip(got, want) for a, b in zip(g, v)), turn
    for a, b in zip(*worlds):
        (a if a.element_size() > 1 else a.view(torch.uint8)).copy_(b if b.element_size() > 1 else b.view(torch.uint8))
    got = call(worlds[0])
    assert torch.equal(got[0], want[1][0]) and torch.equal(got[1], want[1][1])
