"""Paged attention against the fp64 oracle, element by element, with the bounds
the oracle derives from the roundings to bf16 (oracle/operators.py)."""

import numpy as np
import pytest
import torch

import block_sparse_attention_bwd_b200 as sp
from oracle import operators as R

pytestmark = pytest.mark.gpu


class Setup:
    """A pool with the sequences' pages in random order, everything else NaN, and the call's tensors."""

    def __init__(self, lens, heads, kv_heads, head_dim, page_slots, seed=0, heads_first=False, spare=2, **kw):
        self.lens, self.D, self.H, self.Hk, self.ps = lens, head_dim, heads, kv_heads, page_slots
        rng = np.random.default_rng(seed)
        need = [-(-kv // page_slots) for _, kv in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        width = max(need + [1]) + 1
        self.table = np.full((len(lens), width), -1, np.int64)  # entries behind a sequence's pages are never read
        gen = torch.Generator().manual_seed(seed)
        self.rows = []
        k = torch.full((self.pages, page_slots, kv_heads, head_dim), float("nan"), dtype=torch.bfloat16)
        v = k.clone()
        at = 0
        for i, (_, kv) in enumerate(lens):
            mine = order[at:at + need[i]]
            at += need[i]
            self.table[i, :need[i]] = mine
            a, b = (torch.randn((kv, kv_heads, head_dim), generator=gen).bfloat16() for _ in range(2))
            if kw.get("lift"):
                a[:, :, 0] = torch.where(torch.arange(kv) < kv // 16, 8.0, -8.0)[:, None]
            for j, p in enumerate(mine):
                n = min(page_slots, kv - j * page_slots)
                k[p, :n], v[p, :n] = a[j * page_slots:j * page_slots + n], b[j * page_slots:j * page_slots + n]
            self.rows.append((a.double().numpy(), b.double().numpy()))
        if heads_first:  # [kv_heads, slots, D] storage
            k, v = (x.permute(2, 0, 1, 3).contiguous().cuda().permute(1, 2, 0, 3) for x in (k, v))
        self.k, self.v = k.cuda(), v.cuda()
        self.T = sum(q for q, _ in lens) + 3  # rows behind the last sequence
        self.q = (torch.randn((self.T, heads, head_dim), generator=gen) * 1.5).bfloat16().cuda()
        if kw.get("lift"):
            self.q[:, :, 0] = torch.tensor([96.0, -96.0, 0.0]).cuda()[torch.arange(self.T).cuda() % 3][:, None]
        self.d_table = torch.from_numpy(self.table.astype(np.int32)).cuda()
        self.q_start = torch.tensor(np.cumsum([0] + [q for q, _ in lens]), dtype=torch.int32).cuda()
        self.kv_len = torch.tensor([kv for _, kv in lens], dtype=torch.int32).cuda()
        self.cap = kw.get("softcap", 0.0)
        self.slopes = kw.get("slopes")
        self.plan = sp.PagedPlan(heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_slots=page_slots,
                                 max_seqs=kw.get("max_seqs", max(1, len(lens))),
                                 max_q=kw.get("max_q", max([q for q, _ in lens] + [1])),
                                 max_kv=kw.get("max_kv", max([kv for _, kv in lens] + [1])), softcap=self.cap,
                                 slopes=None if self.slopes is None else torch.tensor(self.slopes).float().cuda())

    def run(self, **kw):
        o = torch.full((self.T, self.H, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.T, self.H), 7.0, device="cuda")
        sp.spattn_paged_fwd(kw.get("q", self.q), self.k, self.v, self.d_table, self.q_start, self.kv_len, self.plan,
                            o=o, lse=lse, **{n: x for n, x in kw.items() if n != "q"})
        return o, lse

    def check(self, o, lse):
        o, lse, q = o.cpu().double().numpy(), lse.cpu().double().numpy(), self.q.cpu().double().numpy()
        at = 0
        scale = 1.0 / np.sqrt(self.D)
        slopes = None if self.slopes is None else np.float32(self.slopes).astype(float)
        for (n, kv), (k, v) in zip(self.lens, self.rows):
            if n:
                w, wl, t, tl = R.paged(q[at:at + n], k, v, kv, scale, self.cap, slopes)
                for got, want, tol in ((o[at:at + n], w, t), (lse[at:at + n], wl, tl)):
                    assert np.isfinite(got).all()
                    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / np.maximum(tol, 1e-30)).max())
            at += n
        assert (o[at:] == 7.0).all() and (lse[at:] == 7.0).all()
        sp.spattn_paged_check(self.plan)


CASES = [
    # lens, heads, kv heads, D, page slots, options
    ([(1, 1)], 1, 1, 64, 16, {}),
    ([(1, 777)], 16, 4, 128, 16, dict(softcap=30.0)),
    ([(1, 17), (1, 64), (1, 65), (1, 1), (1, 300)], 8, 8, 128, 64, {}),
    ([(1, 500), (1, 2000), (1, 63)], 32, 4, 64, 48, dict(softcap=4.0, slopes=[0.1 * 0.8 ** i for i in range(32)])),
    ([(5, 5), (130, 200), (0, 0), (1, 99), (0, 40)], 6, 2, 128, 32, {}),
    ([(77, 1000), (3, 15)], 4, 4, 64, 16, dict(slopes=[0.5, 0.01, 0.0, -0.02])),
    ([(40, 700), (1, 90)], 10, 2, 128, 128, dict(softcap=20.0, slopes=[0.3, 0.1, 0.0, -0.01, 0.2] * 2)),
    ([(300, 1500)], 4, 1, 64, 64, dict(softcap=90.0, slopes=[0.01] * 4)),
    ([(33, 3000)], 3, 1, 128, 80, dict(softcap=15.0)),
    ([(1, 5000)], 40, 1, 128, 16, {}),
    ([(2, 2), (2, 3)], 64, 2, 64, 256, dict(softcap=50.0)),
    ([(600, 600)], 2, 2, 128, 16, {}),
]


@pytest.mark.parametrize("lens,heads,kv_heads,d,ps,kw", CASES)
def test_paged_parity(lens, heads, kv_heads, d, ps, kw):
    s = Setup(lens, heads, kv_heads, d, ps, **kw)
    s.check(*s.run())


@pytest.mark.parametrize("lens,heads,kv_heads,d,ps,kw", [
    ([(1, 1)], 1, 1, 64, 16, {}),
    ([(1, 5000)], 2, 1, 64, 32, {}),
    ([(1, 5000)], 2, 1, 64, 32, dict(slopes=[0.02, 0.01])),
    ([(1, 5000)], 2, 1, 64, 32, dict(slopes=[0.0203, 0.019], softcap=55.0)),
    ([(7, 900), (1, 40), (0, 0), (2, 65)], 4, 2, 64, 16, dict(slopes=[0.0, 0.05, -0.05, 0.1])),
    ([(150, 333)], 3, 3, 128, 48, dict(softcap=250.0)),
    ([(65, 2000)], 4, 1, 128, 64, {}),
])
def test_extreme_scores(lens, heads, kv_heads, d, ps, kw):
    """Scores raised by up to 96 (68 for head_dim 128) for the first sixteenth of the keys and lowered for
    the rest, in a third of the rows; the other way round in another third.  Scores that count stay below 2^7,
    for which the oracle's fp32 share (2^-24 * 2^7 * 8 = 2^-14 of a weight) holds; the biases make the
    splits' references differ by as much."""
    s = Setup(lens, heads, kv_heads, d, ps, lift=True, **kw)
    s.check(*s.run())


@pytest.mark.parametrize("max_q,max_kv,max_seqs", [(1, 2000, 3), (9, 2000, 3), (300, 100000, 40), (64, 1 << 20, 3)])
def test_bounds_do_not_change_results(max_q, max_kv, max_seqs):
    """Loose bounds choose other tiles and splits."""
    s = Setup([(1, 1999), (1, 64), (1, 130)], 8, 2, 128, 32, max_q=max_q, max_kv=max_kv, max_seqs=max_seqs, softcap=25.0)
    s.check(*s.run())


def test_strided_cache_and_queries():
    s = Setup([(9, 333), (1, 50)], 6, 3, 64, 32, heads_first=True, slopes=[0.1, 0.2, 0.3, 0.0, 0.05, 0.4])
    s.check(*s.run())
    wide = torch.zeros((s.T, 10, 72), dtype=torch.bfloat16, device="cuda")
    view = wide[:, 2:8, 8:]  # 16-byte aligned rows inside wider ones
    view.copy_(s.q)
    s.check(*s.run(q=view))


def test_workspace_stream_capture_and_new_lengths():
    s = Setup([(1, 900), (1, 3000)], 8, 2, 128, 64, max_kv=4000)
    s.check(*s.run())
    need = s.plan.workspace_bytes(2)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    s.check(*s.run(workspace=ws))
    with pytest.raises(sp.SpattnError):
        s.run(workspace=ws[:-16])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = s.run(stream=side)
    side.synchronize()
    s.check(o, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = s.run()
    # new lengths and tables between replays
    t = Setup([(1, 333), (1, 2999)], 8, 2, 128, 64, seed=5, max_kv=4000, spare=s.pages - 53)  # 6 + 47 pages in use
    assert t.pages == s.pages and t.table.shape[1] <= s.table.shape[1]
    for a, b in ((s.k, t.k), (s.v, t.v), (s.q, t.q), (s.kv_len, t.kv_len)):
        a.copy_(b)
    s.d_table[:, :t.table.shape[1]] = t.d_table
    g.replay()
    torch.cuda.synchronize()
    t.check(o, lse)


def test_two_calls_at_once_with_one_handle():
    s = Setup([(1, 4000)], 16, 2, 128, 16, softcap=30.0)
    want = s.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [s.run(stream=st) for _ in range(10) for st in streams]
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    s.check(*want)


def test_bad_lengths_and_pages_are_reported():
    def status(s):
        o, lse = s.run()
        with pytest.raises(sp.SpattnError) as e:
            sp.spattn_paged_check(s.plan)
        assert e.value.status == sp.SPATTN_ERR_DEVICE
        sp.spattn_paged_check(s.plan)  # reported once
        return o, lse

    lens = [(2, 100), (1, 40)]
    for change in (lambda s: s.kv_len.copy_(torch.tensor([101, 40])),  # beyond max_kv
                   lambda s: s.kv_len.copy_(torch.tensor([1, 40])),  # shorter than its new tokens
                   lambda s: s.kv_len.copy_(torch.tensor([-5, 40])),
                   lambda s: s.q_start.copy_(torch.tensor([-1, 2, 3])),
                   lambda s: s.q_start.copy_(torch.tensor([3, 2, 3]))):
        s = Setup(lens, 4, 2, 64, 16)
        change(s)
        o, lse = status(s)
        # the other sequence is served (rows 2 ..), the rejected one's rows are left alone
        w, _, tol, _ = R.paged(s.q[2:3].cpu().double().numpy(), *s.rows[1], 40, 0.125)
        assert (np.abs(o[2:3].cpu().double().numpy() - w) <= tol).all() and (o[:2] == 7.0).all()
    s = Setup(lens, 4, 2, 64, 16)
    s.q_start.copy_(torch.tensor([0, 2, 900]))  # rows behind q
    status(s)
    for page in (-1, 10 ** 9, -2 ** 31):
        s = Setup(lens, 4, 2, 64, 16)
        s.d_table[0, 3] = page
        s.k[0], s.v[0] = 0.0, 0.0
        status(s)


def test_refusals():
    ok = dict(heads=4, kv_heads=2, head_dim=64, page_slots=16, max_seqs=2, max_q=4, max_kv=64)
    s = Setup([(3, 20)], 4, 2, 64, 16)
    args = [s.q, s.k, s.v, s.d_table, s.q_start, s.kv_len]
    for i, bad in ((0, s.q.float()), (0, s.q[:, :3]), (0, s.q.transpose(0, 1)), (0, s.q.cpu()), (1, s.k[:, :8]),
                   (1, s.k.half()), (2, s.v[:-1]), (1, torch.cat([s.k, s.k], 1)[:, :16]), (3, s.d_table.long()),
                   (3, s.d_table[0]), (4, s.q_start[:-1]), (5, s.kv_len.long()), (5, s.kv_len.cpu())):
        a = list(args)
        a[i] = bad
        with pytest.raises(ValueError):
            sp.spattn_paged_fwd(*a, s.plan)
    with pytest.raises(sp.SpattnError):  # rows off the 16-byte grid
        q = torch.zeros((s.T, 4, 68), dtype=torch.bfloat16, device="cuda")[:, :, 4:]
        sp.spattn_paged_fwd(q, *args[1:], s.plan)
    with pytest.raises(sp.SpattnError):  # more sequences than the handle allows
        sp.spattn_paged_fwd(s.q, s.k, s.v, s.d_table.repeat(2, 1), torch.zeros(3, dtype=torch.int32).cuda(),
                            s.kv_len.repeat(2), s.plan)
    plan = sp.PagedPlan(**ok)
    o, lse = sp.spattn_paged_fwd(s.q, s.k, s.v, s.d_table[:0], s.q_start[:1], s.kv_len[:0], plan)
    assert o.shape == s.q.shape
    s.check(*s.run())
