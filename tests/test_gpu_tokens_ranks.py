"""The token sort's ranks in each of the ways that it counts them (small batches, chunk
counts, the layer's routing kernels) and at their borders, and tokens with many
choices: integers exactly."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


# (T, k, E): 6144 and 16384 slots are the last of small batches, 12288 chunk counts
# the last that are added up; chunks of 256 slots that end inside a token
@pytest.mark.parametrize("T,k,E", [(1, 512, 40), (2, 300, 512), (9, 512, 3), (767, 8, 96), (768, 8, 96), (769, 8, 96),
                                   (2048, 8, 97), (2049, 8, 97), (1366, 9, 48), (8192, 8, 48), (8193, 8, 48),
                                   (50, 256, 16), (30, 257, 16), (100, 100, 1), (4001, 7, 11), (70001, 3, 2),
                                   (131072, 8, 24), (200003, 5, 512)])
def test_ranks(nv, T, k, E):
    import torch
    g = np.random.RandomState(T + k + E)
    ids = g.randint(-1, E + 1, (T, k)).astype(np.int32)
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")[:ok.sum()]
    row = np.full(T * k, -1, np.int32)
    row[order] = np.arange(len(order), dtype=np.int32)
    x = torch.arange(T, device="cuda", dtype=torch.float32).view(T, 1)
    rows = torch.full((T * k, 1), -5.0, device="cuda")
    _, off, got = nv.sort_tokens(x, torch.from_numpy(ids).cuda(), E, rows=rows)
    assert (got.cpu().numpy().reshape(-1) == row).all()
    counts = np.bincount(flat[ok], minlength=E)
    assert (off.cpu().numpy() == np.concatenate([[0], np.cumsum(counts)])).all()
    want = np.full(T * k, -5.0, np.float32)
    want[:len(order)] = order // k
    assert (rows.cpu().numpy().reshape(-1) == want).all()


def test_a_workspace_of_the_asked_size(nv):
    """Nothing is written before or behind it."""
    import torch
    for T, k, E in ((8, 8, 48), (4096, 8, 48), (8193, 8, 48)):
        ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
        x = torch.randn((T, 8), device="cuda")
        n = nv._lib.nvfp4_sort_tokens_workspace(T, E, k)
        buf = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        a = nv.sort_tokens(x, ids, E, workspace=buf[256:256 + n])
        assert bool((buf[:256] == 0x5A).all()) and bool((buf[256 + n:] == 0x5A).all())
        b = nv.sort_tokens(x, ids, E)
        assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("T,k,H", [(200, 40, 8192), (401, 17, 5000), (30, 250, 4100)])
def test_work_groups_that_share_tokens(nv, T, k, H):
    """Few tokens of many choices: several work-groups move a token's row and rank its
    slots, each by itself."""
    import torch
    E = 48
    g = np.random.RandomState(T)
    ids = torch.from_numpy(g.randint(0, E, (T, k)).astype(np.int32)).cuda()
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    order = torch.sort(ids.view(-1).long(), stable=True).indices
    for _ in range(20):
        rows, _, row = nv.sort_tokens(x, ids, E)
        assert torch.equal(rows, x[order // k])
        assert torch.equal(row.view(-1)[order], torch.arange(T * k, device="cuda", dtype=torch.int32))


def test_more_tokens_than_work_groups(nv):
    """2^22 tokens and a few: every one is reached."""
    import torch
    T, H = (1 << 22) + 5, 8
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    x = torch.randint(-100, 100, (T, H), device="cuda").to(torch.bfloat16)
    rows, off, row = nv.sort_tokens(x, ids, 1)
    assert off.tolist() == [0, T] and torch.equal(rows, x)
    w = torch.full((T, 1), 2.0, device="cuda")
    assert torch.equal(nv.unsort_tokens(rows, row, w), 2 * x) and torch.equal(nv.sort_tokens_backward(rows, row), x)
    d_rows, dw = nv.unsort_tokens_backward(x, rows, row, w)
    assert torch.equal(d_rows, 2 * x) and torch.equal(dw[:, 0], (x.float() ** 2).sum(1))
    d = nv.route_topk_backward(w, ids, torch.full((T, 1), 0.5, device="cuda"), 1)
    assert bool((d == 0.5).all())                    # 0.5 * (2 - 0.5 * 2)
