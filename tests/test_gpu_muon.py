"""GPU parity of the Muon step against the float64 oracle (singular value decomposition).

Tolerances: m is one fused multiply-add, 2^-24 relative to |momentum m| + |g|.  The orthogonal
update: a relative error d of the Gram matrix moves the factor of a singular value by at most
sum_j (|b| / a) a^(2 j) d over the steps of one run: 1.39 (1 + 11.9) d = 18 d for the two of
the first, 1.39 (1 + 11.9 + 141) d = 213 d for the three of a later one.  The fp32 sums of
short runs keep d at about 1e-7 (they add up few numbers a thread and then halve): 2.3e-5 in
relative L2, taken as 2.5e-5.  That is against the Newton-Schulz steps of u as float32 holds
it: rounding u (2^-24 of its norm) by itself moves what five steps make of a weak direction by
up to a^5 2^-24 = 2.9e-5, whatever computes them, so the reference takes m from the step (it
is checked by itself) and rounds u once.
"""
import numpy as np
import pytest

from oracle import ops
from tests.helpers import errors, host

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.7750, 2.0315)
UPDATE_REL = 2.5e-5


def matrix(rs, rows, cols, fall):
    """Singular values that fall by 10^fall."""
    side = min(rows, cols)
    left = rs.normal(size=(rows, side)) * np.logspace(0, -fall, side)
    return (left @ rs.normal(size=(side, cols)) / np.sqrt(side)).astype(np.float32)


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def reference(p, g, m_after, momentum, lr, wd, steps, nesterov, scale):
    """p after the step, from the momentum that the step left."""
    mu = np.float64(np.float32(momentum))
    u = (g.astype(np.float64) + mu * m_after).astype(np.float32).astype(np.float64) if nesterov else m_after
    norm = np.linalg.norm(u) + 1e-7
    return p - lr * (wd * p + scale * ops.newton_schulz(u / norm, COEF, steps))


def check_step(lib, shapes, steps=5, nesterov=True, momentum=0.95, fall=2.0, wd=0.0, lr=1.0, zero_p=True, lr_mults=None,
               scales=None, seed=0):
    import torch
    rs = np.random.default_rng(seed + sum(r * 7 + c for r, c in shapes))
    g = [matrix(rs, r, c, fall) for r, c in shapes]
    m = [matrix(rs, r, c, fall) for r, c in shapes]
    p = [np.zeros((r, c), np.float32) if zero_p else rs.normal(0, 0.02, (r, c)).astype(np.float32) for r, c in shapes]
    tp, tg, tm = ([dev(x) for x in xs] for xs in (p, g, m))
    mats = lib.muon_mats(tp, tg, tm, lr_mults, scales)
    cfg = lib.muon_cfg(lr, momentum, wd, 1e-7, COEF, steps, nesterov)
    ws = lib.muon_workspace(mats)
    ws.random_(0, 255)                     # only its status block has to be zero
    ws[:256] = 0
    lib.muon(mats, cfg, ws)
    torch.cuda.synchronize()
    for i, (r, c) in enumerate(shapes):
        if r == 0 or c == 0:
            continue
        mult = 1.0 if lr_mults is None else lr_mults[i]
        scale = np.sqrt(max(1.0, r / c)) if scales is None else scales[i]
        _, rm = ops.muon(p[i], g[i], m[i], lr * mult, momentum, wd, 1e-7, COEF, steps, nesterov, scale)
        rp = reference(p[i].astype(np.float64), g[i], host(tm[i]), momentum, lr * mult, wd, steps, nesterov, scale)
        assert np.all(np.abs(host(tm[i]) - rm) <= 2.0 ** -23 * (momentum * np.abs(m[i]) + np.abs(g[i])) + 1e-30)
        rel, _ = errors(host(tp[i]), rp)
        assert np.all(np.isfinite(host(tp[i]))) and rel <= UPDATE_REL, (i, r, c, rel)
        assert np.array_equal(host(tg[i]), g[i])


@pytest.mark.parametrize("shape", [(1, 1), (1, 5), (9, 1), (2, 3), (5, 1001), (999, 33), (16, 2560), (4096, 16), (8, 8),
                                   (64, 64), (63, 65), (64, 2560), (1024, 64), (33, 257), (17, 513), (1000, 24), (7, 9728)])
@pytest.mark.parametrize("fall", [0.0, 2.0])
def test_muon_shapes(lib, shape, fall):
    check_step(lib, [shape], fall=fall)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("nesterov", [False, True])
def test_muon_steps(lib, steps, nesterov):
    check_step(lib, [(16, 700), (300, 40)], steps=steps, nesterov=nesterov)


def test_muon_hyperparameters(lib):
    check_step(lib, [(16, 500), (900, 16), (20, 30)], lr=0.02, wd=0.1, zero_p=False, lr_mults=[1.0, 16.0, 0.5],
               scales=[0.2, 3.0, 1.0], momentum=0.0)


def test_muon_many_matrices(lib):
    """More matrices than one launch takes, of every rank class, empty ones among them."""
    shapes = [(4, 40 + i % 7) for i in range(300)] + [(60, 70), (0, 5), (3, 0), (20, 90), (100, 12)]
    check_step(lib, shapes)


def test_muon_long(lib):
    check_step(lib, [(64, 70001), (500003, 5)])


def test_muon_zero_update_and_weak_directions(lib):
    import torch
    p, g, m = torch.ones(16, 300, device="cuda"), torch.zeros(16, 300, device="cuda"), torch.zeros(16, 300, device="cuda")
    for eps in (0.0, 1e-7):
        mats = lib.muon_mats([p], [g], [m])
        lib.muon(mats, lib.muon_cfg(0.1, weight_decay=0.5, eps=eps), lib.muon_workspace(mats))
    # two decays by 0.95, each rounded
    assert float((p - 0.95 ** 2).abs().max()) <= 2.0 ** -22
    g[3] = 2.0                                               # a single direction of 16
    q = torch.zeros_like(g)
    mats = lib.muon_mats([q], [g], [m])
    lib.muon(mats, lib.muon_cfg(1.0), lib.muon_workspace(mats))
    ref, _ = ops.muon(0 * host(g), host(g), 0 * host(g), 1.0, 0.95, 0.0, 1e-7, COEF, 5, True, 1.0)
    rel, _ = errors(host(q), ref)
    assert rel <= UPDATE_REL
    assert float(q[:3].abs().max()) == 0 and float(q[4:].abs().max()) == 0


def test_muon_nan_stays_in_its_matrix(lib):
    import torch
    ps, gs, ms = ([torch.randn(8, 100, device="cuda") for _ in range(3)] for _ in range(3))
    gs[1][2, 5] = float("nan")
    mats = lib.muon_mats(ps, gs, ms)
    lib.muon(mats, lib.muon_cfg(0.1), lib.muon_workspace(mats))
    assert bool(torch.isfinite(ps[0]).all() and torch.isfinite(ps[2]).all()) and bool(torch.isnan(ps[1]).any())


@pytest.mark.parametrize("rows,cols", [(16, 500), (500, 16), (15, 501), (501, 15)])
def test_muon_misaligned_repeats_and_graphs(lib, rows, cols):
    """4-byte alignment, untouched neighbours, the same bits again, on another stream and in
    two captured graphs that share a workspace."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rows)
    n = rows * cols
    base = [torch.randn(n + 8, generator=gen, device="cuda") for _ in range(3)]

    def fresh(shift):
        bufs = [torch.full((n + 8,), 7.0, device="cuda") for _ in base]
        views = [b[shift:shift + n] for b in bufs]
        for v, s in zip(views, base):
            v.copy_(s[:n])
        return bufs, [v.view(rows, cols) for v in views]

    cfg = lib.muon_cfg(0.1, weight_decay=0.01)
    results = []
    side = torch.cuda.Stream()
    for shift in (0, 0, 1, 3):
        bufs, v = fresh(shift)
        mats = lib.muon_mats([v[0]], [v[1]], [v[2]])
        ws = lib.muon_workspace(mats)
        side.wait_stream(torch.cuda.current_stream())
        lib.muon(mats, cfg, ws, stream=side if len(results) == 1 else None)
        torch.cuda.synchronize()
        assert all(bool((b[:shift] == 7.0).all()) and bool((b[shift + n:] == 7.0).all()) for b in bufs)
        results.append([x.clone() for x in v])
    assert all(torch.equal(a, b) for a, b in zip(results[0], results[1]))
    for other in results[2:]:                                # element by element the same arithmetic
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
    graphs, outs = [], []
    ws = None
    for _ in range(2):
        _, v = fresh(0)
        mats = lib.muon_mats([v[0]], [v[1]], [v[2]])
        ws = lib.muon_workspace(mats) if ws is None else ws
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            lib.muon(mats, cfg, ws)
        graphs.append((graph, v, mats))
    for graph, v, _ in graphs:
        graph.replay()
        outs.append(v)
    torch.cuda.synchronize()
    for v in outs:
        assert all(torch.equal(a, b) for a, b in zip(results[0], v))


@pytest.mark.parametrize("rows,cols,copies", [(64, 110000, 4), (90001, 40, 4), (64, 2560, 150)])
def test_muon_beside_others(lib, rows, cols, copies):
    """The same bits for a matrix by itself and beside others, where a block takes several of its
    column tiles: their Gram matrices are summed tile by tile either way."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    one = [torch.randn(rows, cols, generator=gen, device="cuda") * 0.02 for _ in range(3)]
    cfg = lib.muon_cfg(0.02, 0.95, 0.1, 1e-7, COEF, 5, True)
    many = [[x.clone() for _ in range(copies)] for x in one]
    for lists in ([[x] for x in one], many):
        mats = lib.muon_mats(*([lists[k] for k in range(3)]))
        lib.muon(mats, cfg, lib.muon_workspace(mats))
    for k in (0, 2):
        assert all(torch.equal(one[k], x) for x in many[k])


@pytest.mark.parametrize("steps", [1, 5])
def test_muon_mixed_shapes_together(lib, steps):
    """Long matrices of ranks above 32 share blocks with others of another rank, side or alignment,
    one of them full of NaN: the same bits as each by itself."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(6)
    shapes = [(64, 2560), (40, 3001), (2999, 33), (4096, 64), (50, 2100), (3500, 52), (63, 2049)] * 9
    sets = [[torch.randn(s, generator=gen, device="cuda") * 0.02 for _ in range(3)] for s in shapes]
    sets[3][1].fill_(float("nan"))
    cfg = lib.muon_cfg(0.02, 0.95, 0.1, 1e-7, COEF, steps, True)
    alone = [[x.clone() for x in xs] for xs in sets]
    for xs in alone:
        mats = lib.muon_mats(*([x] for x in xs))
        lib.muon(mats, cfg, lib.muon_workspace(mats))
    mats = lib.muon_mats(*([xs[k] for xs in sets] for k in range(3)))
    ws = lib.muon_workspace(mats)
    ws[256:].fill_(255)                                       # NaN in whatever is read unwritten
    lib.muon(mats, cfg, ws)
    for i, (xs, ys) in enumerate(zip(sets, alone)):
        assert bool(torch.isnan(xs[0]).any()) == (i == 3)
        for k in (0, 2):
            assert torch.equal(xs[k].nan_to_num(7.0), ys[k].nan_to_num(7.0)), (i, shapes[i])
    lib.workspace_status(ws)


def test_muon_refusals(lib):
    import torch
    z = lambda *s: torch.zeros(*s, device="cuda")
    with pytest.raises(ValueError, match="twice"):
        a = z(4, 4)
        lib.muon_mats([a, a], [z(4, 4), z(4, 4)], [z(4, 4), z(4, 4)])
    with pytest.raises(ValueError, match="also a param"):
        a = z(4, 4)
        lib.muon_mats([a], [a], [z(4, 4)])
    with pytest.raises(ValueError, match="length"):
        lib.muon_mats([z(4, 4)], [], [z(4, 4)])
    with pytest.raises(ValueError, match="one shape"):
        lib.muon_mats([z(4, 4)], [z(4, 5)], [z(4, 4)])
    with pytest.raises(ValueError, match="contiguous"):
        lib.muon_mats([z(4, 5)], [z(5, 4).t()], [z(4, 5)])
    with pytest.raises(TypeError):
        lib.muon_mats([z(4, 5).bfloat16()], [z(4, 5)], [z(4, 5)])
    mats = lib.muon_mats([z(65, 66)], [z(65, 66)], [z(65, 66)])
    with pytest.raises(lib.TlbError, match="at most 64"):
        lib.muon(mats, lib.muon_cfg(0.1), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    mats = lib.muon_mats([z(8, 66)], [z(8, 66)], [z(8, 66)])
    with pytest.raises(lib.TlbError, match="workspace"):
        lib.muon(mats, lib.muon_cfg(0.1), torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lib.TlbError, match="steps"):
        lib.muon(mats, lib.muon_cfg(0.1, steps=0), lib.muon_workspace(mats))
    none = lib.muon_mats([], [], [])
    lib.muon(none, lib.muon_cfg(0.1), lib.muon_workspace(none))
