"""A serving step on the paged FP8 cache where its parts meet: block tables, slots, the write and attention."""
import numpy as np
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
from paged_ref import encode, page_tables

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def sums(lens):
    return [0] + np.cumsum(lens).tolist()


def test_pages_whose_slots_do_not_fit_an_int():
    """Entries so large that page * page_size wraps are no pages: their slots are -1, not another page's."""
    for P in (16, 128):
        wrap = (1 << 32) // P                                 # times P: 0 in 32 bits
        top = ((1 << 31) - 1) // P                            # the last page whose slots fit
        table = i32([[3, wrap, -1, -1], [wrap // 2, -1, -1, -1], [top, -1, -1, -1]])
        got = qz.qz_block_tables(i32([P + 2, 1, P - 1]), i32([P, 1, 2]), table, i32([wrap, top, 5]), i32([0]), P, P + 4)
        slots = [-1] * P + [-1] + [top * P + P - 1, top * P, -1]
        assert got[0].tolist() == slots


def serving_step(s, ws):
    """One step on static inputs: tables, write, attention over `s["T"]` slots."""
    slots, pos, cu, kv, head = qz.qz_block_tables(s["ctx"], s["new"], s["table"], s["free"], s["head"], 16, s["T"])
    qz.qz_kv_append_fp8_paged(s["qkv"][:, 8:10], s["qkv"][:, 10:], slots, s["cache"])
    out, lse = qz.qz_attn_fp8_paged(s["qkv"][:, :8], s["cache"], s["table"], kv, cu, s["T"], 0.125, ws=ws, lse=True)
    return slots, pos, cu, kv, head, out, lse


def serving_state(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, T, pages, D = 5, 210, 60, 64
    s = dict(T=T, ctx=i32([0] * B), new=i32([0] * B), head=i32([0]), free=torch.randperm(pages, generator=g, device="cuda").to(torch.int32),
             table=torch.full((B, 40), -1, dtype=torch.int32, device="cuda"), cache=qz.PagedKV.empty(pages, 2, 16, D),
             qkv=torch.empty((T, 12, D), dtype=torch.bfloat16, device="cuda"))
    s["cache"].k_codes.zero_()
    s["cache"].v_codes.zero_()
    steps = []
    for new in ([70, 1, 130, 0, 9], [1, 1, 1, 100, 1], [1, 0, 1, 1, 1], [50, 1, 1, 1, 40]):
        steps.append((new, torch.randn((T, 12, D), generator=g, device="cuda").to(torch.bfloat16)))
    return s, steps


def play(s, steps, run):
    """The steps' outputs, rows of the requests only, and the cache in the end."""
    got = []
    for new, qkv in steps:
        s["new"].copy_(i32(new))
        s["qkv"].copy_(qkv)
        slots, pos, cu, kv, head, out, lse = run()
        n = sum(new)
        got += [slots.clone(), pos.clone(), cu.clone(), kv.clone(), head.clone(), out[:n].clone(), lse[:n].clone()]
        s["ctx"].copy_(kv)
        s["head"].copy_(head)
    return got + [s["table"].clone()] + [x.clone() for x in (s["cache"].k_codes, s["cache"].v_codes)]


def test_a_step_in_a_graph():
    """Tables, write and attention captured once and replayed on other lengths: the bits of the calls themselves."""
    s, steps = serving_state(0)
    ws = qz.Workspace()
    want = play(s, steps, lambda: serving_step(s, ws))
    s, steps = serving_state(0)
    ws.get(qz.qz_workspace_size(qz.OP_ATTN_FP8_PAGED, s["T"] * 4, 64))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outputs = serving_step(s, ws)

    def replay():
        graph.replay()
        return outputs
    got = play(s, steps, replay)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_streams_at_once():
    """Calls of all kinds on two streams that run beside one another, a workspace each."""
    sets = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        P, D, H = 32, 128, 4
        k, v = (encode(torch.randn((300, H, P, D), generator=g, device="cuda")) for _ in range(2))
        cache, jobs = qz.PagedKV(k[0], v[0], k[1], v[1]), []
        for kv, n in (([2000], [1]), ([700, 900, 30], [700, 1, 5]), ([2500], [300]), ([400] * 20, [3] * 20), ([640] * 12, [200] * 12)):
            table, _ = page_tables(kv, P, 300 - sum(-(-x // P) for x in kv), g)
            jobs.append((torch.randn((sum(n), 4 * H, D), generator=g, device="cuda").to(torch.bfloat16), cache, table, i32(kv),
                         i32(sums(n)), max(n), 0.1))
        sets.append((jobs, [qz.qz_attn_fp8_paged(*j)[0] for j in jobs], qz.Workspace(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for r in range(6):
        for i, (jobs, _, ws, st) in enumerate(sets):
            with torch.cuda.stream(st):
                outs[i] += [qz.qz_attn_fp8_paged(*j, ws=ws)[0] for j in jobs[r % 5:] + jobs[:r % 5]]
    torch.cuda.synchronize()
    for i, (jobs, alone, _, _) in enumerate(sets):
        for r in range(6):
            for j in range(5):
                assert torch.equal(outs[i][r * 5 + j], alone[(j + r % 5) % 5]), (i, r, j)
    assert qz.qz_device_error() == 0


def test_outputs_belong_to_the_stream_of_the_call():
    """Memory that the current stream has freed but still writes to does not become the output, lse, workspace or slot
    map of a call on another stream."""
    g = torch.Generator(device="cuda").manual_seed(0)
    P, D, H, L = 32, 128, 2, 3000
    k, v = (encode(torch.randn((L // P + 1, H, P, D), generator=g, device="cuda")) for _ in range(2))
    cache, table = qz.PagedKV(k[0], v[0], k[1], v[1]), torch.arange(L // P + 1, dtype=torch.int32, device="cuda")[None]
    side = torch.cuda.Stream()
    for n in (1, 100):
        q = torch.randn((n, 8 * H, D), generator=g, device="cuda").to(torch.bfloat16)
        args = (q, cache, table, i32([L]), i32([0, n]), n, 0.1)
        lens, free, head = (i32([0, 40]), i32([n, 7])), torch.arange(300, dtype=torch.int32, device="cuda"), i32([5])
        tables = [torch.zeros((2, 200), dtype=torch.int32, device="cuda") for _ in range(2)]
        want = qz.qz_attn_fp8_paged(*args, lse=True)
        want += qz.qz_block_tables(*lens, tables[0], free, head, P, n + 7)
        torch.cuda.synchronize()
        need = qz.qz_workspace_size(qz.OP_ATTN_FP8_PAGED, n * 8, D)
        torch.cuda._sleep(100_000_000)                        # the current stream is behind
        for shape, dtype in ((q.shape, torch.bfloat16), (q.shape[:2], torch.float32), ((need,), torch.uint8), ((n + 7,), torch.int32)):
            for _ in range(3):
                torch.empty(shape, dtype=dtype, device="cuda").fill_(7)
        got = qz.qz_attn_fp8_paged(*args, lse=True, stream=side)
        got += qz.qz_block_tables(*lens, tables[1], free, head, P, n + 7, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
