"""Packed attention with grouped heads against its 64-bit form (GB300)."""

import math

import pytest
import torch

from tensor_transformer_mlp_forward_gb300 import binding
from tests import packed_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _cu(lens, start=0):
    cu = [start]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _inputs(T, nh, nkv, d, seed, dense=False):
    """Q, K, V, dO (CPU) and the first three on the GPU as parts of one
    projection's rows with 8 columns more (or dense)."""
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(T, n, d, generator=g).to(BF) for n in (nh, nkv, nkv, nh))
    if dense:
        return (q, k, v, do), [x.cuda() for x in (q, k, v)] + [do.cuda()]
    rows = torch.zeros(T, (nh + 2 * nkv) * d + 8, dtype=BF, device="cuda")
    parts, at = [], 0
    for x in (q, k, v):
        n = x.shape[1] * d
        rows[:, at:at + n] = x.reshape(T, n).cuda()
        parts.append(rows[:, at:at + n].unflatten(1, (x.shape[1], d)))
        at += n
    return (q, k, v, do), parts + [do.cuda()]


def _check_forward(O, lse, cpu, cu, scale):
    q, k, v, _ = cpu
    Or, lr, A = ref.attention(q, k, v, cu, scale)
    rows = slice(cu[0], cu[-1])
    O, lse = O.double().cpu(), lse.double().cpu()
    # P rounded to bf16, O rounded to bf16, exponents of sums of d <= 160 terms
    # in fp32: d 2^-24 times sum |q k| scale log2(e) < 24 is below 2^-12
    tol = 2.0 ** -8 * (1 + 2.0 ** -6) * (A + Or.abs()) + 2.0 ** -11 * A
    assert ((O - Or).abs() <= tol)[rows].all(), ((O - Or).abs() - tol)[rows].max()
    assert ((lse - lr).abs() <= 2.0 ** -11 + 2.0 ** -21 * lr.abs())[:, rows].all()


def _check_backward(got, cpu, o, lse, do, cu, scale):
    q, k, v, _ = cpu
    want, tol = ref.attention_backward(q, k, v, o, lse, do, cu, scale)
    for name, x, w, t in zip(("dQ", "dK", "dV"), got, want, tol):
        err = (x.double().cpu() - w).abs()[cu[0]:cu[-1]]
        assert (err <= t[cu[0]:cu[-1]]).all(), (name, (err - t[cu[0]:cu[-1]]).max())


CASES = [
    # lengths, tokens before and behind them, nh, nkv, d
    ([1], 0, 0, 1, 1, 64),
    ([1, 0, 1, 2, 0], 0, 3, 4, 2, 128),
    ([127, 128, 129], 0, 0, 4, 2, 128),
    ([127, 1, 257], 5, 11, 3, 3, 64),
    ([255, 256, 63], 1, 0, 6, 2, 96),
    ([65, 64, 300], 0, 70, 4, 1, 160),
    ([385], 0, 0, 5, 5, 160),
    ([0, 640, 0], 3, 1, 8, 1, 128),
    ([33] * 9, 0, 0, 2, 2, 96),
    ([200, 511], 0, 0, 12, 4, 64),
    ([700], 0, 0, 3, 1, 128),
]


@pytest.mark.parametrize("lens,before,behind,nh,nkv,d", CASES)
def test_forward_and_backward(lens, before, behind, nh, nkv, d):
    cu = _cu(lens, before)
    T = cu[-1] + behind
    cpu, (q, k, v, do) = _inputs(T, nh, nkv, d, seed=len(lens) * 1000 + T)
    scale = d ** -0.5
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    O = torch.full((T, nh, d), 7.0, dtype=BF, device="cuda")
    lse = torch.full((nh, T), 7.0, device="cuda")
    binding.tp_attn_packed_forward(q, k, v, cud, O=O, lse=lse)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    _check_forward(O, lse, cpu, cu, scale)
    outside = torch.ones(T, dtype=torch.bool, device="cuda")
    outside[cu[0]:cu[-1]] = False
    assert (O[outside] == 7.0).all() and (lse[:, outside] == 7.0).all()

    # the backward pass from the exact O and lse, rounded to their types
    Or, lr, _ = ref.attention(*cpu[:3], cu, scale)
    o, l32 = Or.to(BF), lr.float()
    rows = torch.full((T, (nh + 2 * nkv) * d + 16), 7.0, dtype=BF, device="cuda")
    grads = [rows[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in
             ((0, nh), (nh, nh + nkv), (nh + nkv, nh + 2 * nkv))]
    got = binding.tp_attn_packed_backward(q, k, v, o.cuda(), l32.cuda(), do, cud, dQ=grads[0], dK=grads[1],
                                          dV=grads[2])
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    _check_backward(got, cpu, o, l32, cpu[3], cu, scale)
    assert (rows[outside] == 7.0).all() and (rows[:, (nh + 2 * nkv) * d:] == 7.0).all()


def test_scale_and_large_scores():
    # scores of a few hundred: one key takes all the weight
    cu = [0, 150, 290]
    cpu, (q, k, v, do) = _inputs(290, 4, 2, 64, seed=5, dense=True)
    cpu = (cpu[0] * 4, cpu[1] * 4, cpu[2], cpu[3])  # exact in bf16
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    O, lse = binding.tp_attn_packed_forward(cpu[0].cuda(), cpu[1].cuda(), v, cud, scale=0.5)
    Or, lr, A = ref.attention(*cpu[:3], cu, 0.5)
    # sum |q k| scale log2(e) < 2500 now: 64 2^-24 of it is below 2^-6 of an exponent,
    # 2 ln 2 times that of a weight
    assert ((O.double().cpu() - Or).abs() <= (2.0 ** -7 + 2.0 ** -5) * A).all()
    assert ((lse.double().cpu() - lr).abs() <= 2.0 ** -6).all()


@pytest.mark.parametrize("nh,nkv,d", [(4, 2, 128), (3, 3, 160), (2, 1, 64)])
def test_sequences_keep_their_nan_to_themselves(nh, nkv, d):
    lens = [100, 77, 130, 40]
    cu = _cu(lens, 2)
    T = cu[-1] + 9
    cpu, _ = _inputs(T, nh, nkv, d, seed=8, dense=True)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    clean = [x.clone() for x in cpu]
    Or, lr, _ = ref.attention(*clean[:3], cu, d ** -0.5)
    o, lse = Or.to(BF), lr.float()
    bad = [x.clone() for x in clean]
    for i, x in enumerate(bad):  # sequences 1 and 3 and the rows around all
        fill = (math.nan, math.inf, -math.inf, math.nan)[i]
        x[:cu[0]] = fill
        x[cu[1]:cu[2]] = fill
        x[cu[3]:] = fill
    obad, lbad = o.clone(), lse.clone()
    obad[cu[1]:cu[2]] = math.inf
    lbad[:, cu[3]:] = math.nan
    keep = torch.zeros(T, dtype=torch.bool)
    keep[cu[0]:cu[1]] = keep[cu[2]:cu[3]] = True
    outs = []
    for x, oo, ll in ((clean, o, lse), (bad, obad, lbad)):
        q, k, v, do = (t.cuda() for t in x)
        f = binding.tp_attn_packed_forward(q, k, v, cud)
        b = binding.tp_attn_packed_backward(q, k, v, oo.cuda(), ll.cuda(), do, cud)
        outs.append([f[0][keep.cuda()], f[1][:, keep.cuda()]] + [t[keep.cuda()] for t in b])
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    for a, b in zip(*outs):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_results_repeat_bit_for_bit():
    cu = torch.tensor(_cu([300, 5, 411, 128]), dtype=torch.int32, device="cuda")
    _, (q, k, v, do) = _inputs(844, 8, 2, 128, seed=11)
    first = None
    for _ in range(4):
        O, lse = binding.tp_attn_packed_forward(q, k, v, cu)
        out = [O, lse, *binding.tp_attn_packed_backward(q, k, v, O, lse, do, cu)]
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_equal_sequences_agree_with_the_unpacked_block():
    # the framework's attention of sequences of one length, a head each
    nb, s, nh, d = 3, 200, 4, 128
    T, h = nb * s, nh * d
    _, (q, k, v, do) = _inputs(T, nh, nh, d, seed=21)
    qkv = torch.cat([x.reshape(T, h) for x in (q, k, v)], 1)
    O1, lse1 = binding.tp_attn_core_forward(qkv, nb, nh)
    dqkv = binding.tp_attn_core_backward(qkv, O1, lse1, do.reshape(T, h), nb, nh)
    cu = torch.arange(0, T + 1, s, dtype=torch.int32, device="cuda")
    O2, lse2 = binding.tp_attn_packed_forward(q, k, v, cu)
    g = binding.tp_attn_packed_backward(q, k, v, O2, lse2, do, cu)
    rel = lambda a, b: float((a.double() - b.double()).abs().max() / b.double().abs().max())  # noqa: E731
    assert rel(O2.reshape(T, h), O1) <= 2e-2 and rel(lse2, lse1) <= 1e-4
    for i, x in enumerate(g):
        assert rel(x.reshape(T, h), dqkv[:, i * h:(i + 1) * h]) <= 2e-2


@pytest.mark.parametrize("cu", [[0, 50, 40, 90], [0, 50, 101], [-1, 50, 90], [60, 50]])
def test_bad_offsets_write_nothing(cu):
    _, (q, k, v, do) = _inputs(100, 2, 1, 64, seed=2)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    O = torch.full((100, 2, 64), 7.0, dtype=BF, device="cuda")
    lse = torch.full((2, 100), 7.0, device="cuda")
    binding.tp_attn_packed_forward(q, k, v, cud, O=O, lse=lse)
    assert binding.device_status() == binding.TPMLP_ERR_SHAPE
    assert (O == 7.0).all() and (lse == 7.0).all()
    g = [torch.full((100, n, 64), 7.0, dtype=BF, device="cuda") for n in (2, 1, 1)]
    binding.tp_attn_packed_backward(q, k, v, O, lse, do, cud, dQ=g[0], dK=g[1], dV=g[2])
    assert binding.device_status() == binding.TPMLP_ERR_SHAPE
    assert all((x == 7.0).all() for x in g)
    assert binding.device_status() == 0


def test_many_short_sequences_and_one_cta_planning_them():
    # more sequences than the planning CTA has threads, most of them empty
    g = torch.Generator().manual_seed(31)
    lens = [int(x) for x in torch.randint(0, 4, (2500,), generator=g)]
    cu = _cu(lens)
    cpu, (q, k, v, do) = _inputs(cu[-1], 2, 1, 64, seed=32)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    O, lse = binding.tp_attn_packed_forward(q, k, v, cud)
    _check_forward(O, lse, cpu, cu, 0.125)
    Or, lr, _ = ref.attention(*cpu[:3], cu, 0.125)
    got = binding.tp_attn_packed_backward(q, k, v, Or.to(BF).cuda(), lr.float().cuda(), do, cud)
    _check_backward(got, cpu, Or.to(BF), lr.float(), cpu[3], cu, 0.125)


def test_offsets_past_32_bits():
    # rows whose first value is 2^31 values and more into the matrix
    nh, d, T = 64, 128, 262400
    cu = [T - 200, T - 73, T]
    g = torch.Generator().manual_seed(7)
    small = [torch.randn(200, n, d, generator=g).to(BF) for n in (nh, 1, 1, nh)]
    big = []
    for x in small:
        full = torch.zeros((T,) + tuple(x.shape[1:]), dtype=BF, device="cuda")
        full[T - 200:] = x.cuda()
        big.append(full)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    O, lse = binding.tp_attn_packed_forward(*big[:3], cud)
    rel = [c - (T - 200) for c in cu]
    _check_forward(O[T - 200:], lse[:, T - 200:], small, rel, d ** -0.5)
    got = binding.tp_attn_packed_backward(*big[:3], O, lse, big[3], cud)
    _check_backward([x[T - 200:] for x in got], small, O[T - 200:].cpu(), lse[:, T - 200:].cpu(), small[3], rel,
                    d ** -0.5)


def test_a_long_sequence_of_more_ranks_than_shared_memory_counts():
    # 4096 tiles of 128 and more take the plan's counters in the workspace; the
    # tokens that are looked at are the first and last of the sequence
    T, d = 4096 * 128 + 77, 64
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(T, 1, d, generator=g).to(BF) for _ in range(2))
    q = torch.randn(T, 2, d, generator=g).to(BF)
    cud = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    O, lse = binding.tp_attn_packed_forward(q.cuda(), k.cuda(), v.cuda(), cud)
    for t in (0, 1, 300, T // 2, T - 1):
        z = (k[:t + 1, 0].double() @ q[t].double().t()) * d ** -0.5
        p = torch.softmax(z, 0)
        want, A = p.t() @ v[:t + 1, 0].double(), p.t() @ v[:t + 1, 0].double().abs()
        # l sums up to 2^19 terms in fp32, 128 at a time: 2^12 additions
        assert ((O[t].double().cpu() - want).abs() <= 2.0 ** -8 * (A + want.abs()) + 2.0 ** -10 * A).all(), t
        assert ((lse[:, t].double().cpu() - torch.logsumexp(z, 0) / math.log(2.0)).abs() <= 2.0 ** -9).all()


@pytest.mark.parametrize("nh,nkv,d", [(5, 5, 64), (5, 5, 128), (3, 3, 160), (4, 2, 64)])
def test_ragged_batches_many_times(nh, nkv, d):
    # long and short documents in turn, more items than SMs: warps that skip items run
    # ahead of those that do not
    g = torch.Generator().manual_seed(nh + d)
    lens = [int(n) for n in torch.randint(0, 400, (70,), generator=g)]
    cu = _cu(lens)
    cpu, (q, k, v, do) = _inputs(cu[-1], nh, nkv, d, seed=71)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    O, lse = binding.tp_attn_packed_forward(q, k, v, cud)
    _check_forward(O, lse, cpu, cu, d ** -0.5)
    Or, lr, _ = ref.attention(*cpu[:3], cu, d ** -0.5)
    o, l32 = Or.to(BF), lr.float()
    grads = binding.tp_attn_packed_backward(q, k, v, o.cuda(), l32.cuda(), do, cud)
    _check_backward(grads, cpu, o, l32, cpu[3], cu, d ** -0.5)
    for _ in range(40):
        again = binding.tp_attn_packed_forward(q, k, v, cud)
        assert torch.equal(again[0], O) and torch.equal(again[1], lse)
        again = binding.tp_attn_packed_backward(q, k, v, o.cuda(), l32.cuda(), do, cud)
        assert all(torch.equal(a, b) for a, b in zip(again, grads))


@pytest.mark.parametrize("lens,nh,nkv,d", [([2, 1, 2, 3, 0, 2, 1], 4, 2, 64), ([2], 1, 1, 128), ([5, 2, 9, 64, 127, 128, 3], 6, 2, 96),
                                           ([2, 4, 65, 128, 1, 100], 3, 3, 160), ([3, 128, 40, 2], 16, 1, 128)])
def test_short_sequences_keep_dS_in_two_parts(lens, nh, nkv, d):
    # where a gradient is one or two terms, dS's rounding alone would be as large as the
    # result's: within 128 tokens of a sequence's start nothing of it may be left
    cu = _cu(lens)
    cpu, (q, k, v, do) = _inputs(cu[-1], nh, nkv, d, seed=17 + d)
    Or, lr, _ = ref.attention(*cpu[:3], cu, d ** -0.5)
    o, l32 = Or.to(BF), lr.float()
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = binding.tp_attn_packed_backward(q, k, v, o.cuda(), l32.cuda(), do, cud)
    want, tol = ref.attention_backward(*cpu[:3], o, l32, cpu[3], cu, d ** -0.5, two=True)
    for name, x, w, t in list(zip(("dQ", "dK"), got, want, tol)):
        err = (x.double().cpu() - w).abs()
        assert (err <= t).all(), (name, (err - t).max())
        assert (err.norm() <= 1.1 * (w.to(BF).double() - w).norm() + 2.0 ** -12 * w.norm())


def test_groups_dealt_to_parts():
    # 64 query heads on 8: the dK/dV kernel's items are few, and each group's heads go to
    # parts whose sums are added behind; gradients into parts of one matrix, tokens
    # outside the sequences left alone
    cu = [3, 403, 403, 990]
    T, nh, nkv, d = 1000, 64, 8, 64
    cpu, (q, k, v, do) = _inputs(T, nh, nkv, d, seed=51)
    Or, lr, _ = ref.attention(*cpu[:3], cu, d ** -0.5)
    rows = torch.full((T, (nh + 2 * nkv) * d), 7.0, dtype=BF, device="cuda")
    g = [rows[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, nh), (nh, nh + nkv), (nh + nkv, nh + 2 * nkv))]
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = binding.tp_attn_packed_backward(q, k, v, Or.to(BF).cuda(), lr.float().cuda(), do, cud, dQ=g[0], dK=g[1],
                                          dV=g[2])
    assert binding.last_launch_count() == 4  # delta and plan, dQ, dK and dV, parts
    _check_backward(got, cpu, Or.to(BF), lr.float(), cpu[3], cu, d ** -0.5)
    assert (rows[:3] == 7.0).all() and (rows[990:] == 7.0).all()
    # a workspace, O and gradients that start on 16-byte boundaries only
    need = binding.lib().tp_attn_packed_backward_workspace_bytes(3, T, nh, nkv, d)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]
    odd = [torch.empty(x.numel() + 8, dtype=BF, device="cuda")[8:].view(x.shape) for x in got]
    again = binding.tp_attn_packed_backward(q, k, v, Or.to(BF).cuda(), lr.float().cuda(), do, cud, dQ=odd[0], dK=odd[1],
                                            dV=odd[2], workspace=ws)
    assert all(torch.equal(a[3:990], b[3:990]) for a, b in zip(got, again))
    O = torch.empty(T * nh * d + 8, dtype=BF, device="cuda")[8:].view(T, nh, d)
    binding.tp_attn_packed_forward(q, k, v, cud, O=O)
    assert torch.equal(O[3:990], binding.tp_attn_packed_forward(q, k, v, cud)[0][3:990])


def test_dependent_launch_and_threads_change_nothing():
    import threading

    cu = torch.tensor(_cu([200, 1, 90, 333, 140]), dtype=torch.int32, device="cuda")
    sets = [_inputs(764, 8, 2, 128, seed=60 + i)[1] for i in range(3)]

    def run(x):
        O, lse = binding.tp_attn_packed_forward(*x[:3], cu)
        return [O, lse, *binding.tp_attn_packed_backward(*x[:3], O, lse, x[3], cu)]

    want = [run(x) for x in sets]
    old = binding.set_dependent_launch(0)
    try:
        assert all(torch.equal(a, b) for x, w in zip(sets, want) for a, b in zip(run(x), w))
    finally:
        binding.set_dependent_launch(old)
    torch.cuda.synchronize()
    got, bad = [None] * 3, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = run(sets[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 - reported below
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    assert binding.device_status() == 0


def test_other_stream_and_graph_with_new_lengths():
    T, nh, nkv, d = 400, 4, 2, 128
    cpu, (q, k, v, do) = _inputs(T, nh, nkv, d, seed=41)
    cud = torch.tensor([0, 100, 400], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    O, lse = binding.tp_attn_packed_forward(q, k, v, cud, stream=s)
    s.synchronize()
    _check_forward(O, lse, cpu, [0, 100, 400], d ** -0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, lse = binding.tp_attn_packed_forward(q, k, v, cud)
        grads = binding.tp_attn_packed_backward(q, k, v, O, lse, do, cud)
    eager = []
    for lens in ([100, 300], [399, 1], [0, 400], [250, 150]):
        cu = _cu(lens)
        cud.copy_(torch.tensor(cu, dtype=torch.int32))
        graph.replay()
        other = binding.tp_attn_packed_forward(q, k, v, cud)  # beside the graph's next replay
        graph.replay()
        torch.cuda.synchronize()
        _check_forward(O, lse, cpu, cu, d ** -0.5)
        assert torch.equal(other[0], O) and torch.equal(other[1], lse)
        eager = binding.tp_attn_packed_backward(q, k, v, O, lse, do, cud)
        assert all(torch.equal(a, b) for a, b in zip(eager, grads))
    assert binding.device_status() == 0


def test_binding_refuses():
    _, (q, k, v, _) = _inputs(20, 4, 2, 64, seed=1)
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="strides"):
        binding.tp_attn_packed_forward(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, cu)
    with pytest.raises(ValueError, match="K"):
        binding.tp_attn_packed_forward(q, k.float(), v, cu)
    with pytest.raises(ValueError, match="V has shape"):
        binding.tp_attn_packed_forward(q, k, v[:10], cu)
    with pytest.raises(ValueError, match="cu_seqlens"):
        binding.tp_attn_packed_forward(q, k, v, cu.long())
    with pytest.raises(binding.TpMlpError):
        binding.tp_attn_packed_forward(q[:, :3], k, v, cu)
    with pytest.raises(binding.TpMlpError):
        binding.tp_attn_packed_forward(q, k, v, cu, scale=-1.0)
    empty = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    O, lse = binding.tp_attn_packed_forward(empty, empty[:, :2], empty[:, :2], torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert O.shape == (0, 4, 64) and lse.shape == (4, 0)
