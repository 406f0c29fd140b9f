"""Calls with a stream of their own: what they allocate is that stream's
memory, so no call writes a block that work queued on the current stream
still uses, and two calls at once do not share a workspace."""
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_calls():
    """name -> call(stream), each returning the tensors it allocated."""
    g = torch.Generator("cuda").manual_seed(1)
    T, H, R, bs, nb = 300, 16, 512, 64, 64
    w, c = normal(g, H * 256, R), normal(g, T, R)
    q, o = normal(g, T, H, 192), normal(g, T, H, R)
    kv, k_pe = normal(g, T, H, 256), normal(g, T, 64)
    cu, cache = i32([0, T]), normal(g, nb, bs, R + 64)
    table = i32([list(range(nb))])
    rows, free, count = i32([[-1] * nb]), i32(list(range(nb))), i32([nb])
    new, old = i32([T]), i32([0])
    ql, lens = normal(g, T, H, R + 64), i32([4000] * T)
    tables, parts, lses = table.repeat(T, 1), normal(g, 3, T, H, R), normal(g, 3, T, H).float()
    return {
        "batch_build": lambda s: mla.batch_build(new, old, rows, free, count, bs, nb, T, stream=s),
        "gather_cache": lambda s: mla.gather_cache(cache, table, cu, T, stream=s),
        "expand_kv": lambda s: mla.expand_kv(c, w, H, stream=s),
        "absorb_q": lambda s: (mla.absorb_q(q[..., :128], w, stream=s),),
        "project_v": lambda s: (mla.project_v(o, w, stream=s),),
        "prefill": lambda s: mla.prefill(q, kv[..., :128], kv[..., 128:], k_pe, cu, cu, SCALE,
                                         num_kv_splits=3, stream=s),
        "decode": lambda s: mla.decode(ql, cache, tables, lens, SCALE, 4, stream=s),
        "decode_pair": lambda s: mla.decode((ql[..., :R], ql[..., R:]), cache, tables, lens, SCALE,
                                            4, stream=s),
        "lse_merge": lambda s: mla.lse_merge(parts, lses, stream=s),
    }


NAMES = ["batch_build", "gather_cache", "expand_kv", "absorb_q", "project_v", "prefill",
         "decode", "decode_pair", "lse_merge"]


def wait_inputs(side):
    side.wait_stream(torch.cuda.current_stream())


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_the_launch_streams_memory(cuda_dev, name):
    call = make_calls()[name]
    ref = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    for _ in range(3):
        # blocks of the outputs' sizes, free in the current stream's pool but
        # still to be written by what is queued there
        freed = [torch.empty_like(x) for x in ref]
        torch.cuda._sleep(20_000_000)
        for x in freed:
            x.zero_()
        ptrs = {x.data_ptr() for x in freed}
        del freed, x
        wait_inputs(side)
        out = call(side)
        assert not ptrs & {x.data_ptr() for x in out}
        torch.cuda.synchronize()
        for x, r in zip(out, ref):
            assert torch.equal(x, r)
        del out, x


@pytest.mark.parametrize("name", NAMES)
def test_outputs_used_and_let_go_on_the_current_stream(cuda_dev, name):
    """A block that the current stream still reads is not given out again."""
    call = make_calls()[name]
    ref = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    wait_inputs(side)
    out = call(side)
    ptrs = {x.data_ptr() for x in out}
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    kept = [x.clone() for x in out]  # queued behind the sleep
    del out
    again = call(side)
    assert not ptrs & {x.data_ptr() for x in again}
    torch.cuda.synchronize()
    for x, r in zip(kept, ref):
        assert torch.equal(x, r)


def test_two_split_attentions_on_two_streams(cuda_dev):
    """The first call's workspace is let go when it returns, with its kernels
    still queued; the second runs at once, on its own stream."""
    g = torch.Generator("cuda").manual_seed(2)
    cases = []
    for n, keys in ((40, 9000), (40, 9100)):  # workspaces of one size
        q, kv, kp = normal(g, n, 16, 192), normal(g, keys, 16, 256), normal(g, keys, 64)
        a = (q, kv[..., :128], kv[..., 128:], kp, i32([0, n]), i32([0, keys]), SCALE)
        want = mla.prefill(*a, num_kv_splits=8)
        cases.append((a, want))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        torch.cuda._sleep(1_000_000 * (i % 3))
        got = [mla.prefill(*cases[0][0], num_kv_splits=8),
               mla.prefill(*cases[1][0], num_kv_splits=8, stream=side)]
        torch.cuda.synchronize()
        for (o, lse), (_, want) in zip(got, cases):
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("name", NAMES)
def test_captured_on_a_forked_stream(cuda_dev, name):
    """A call on a stream that joins a capture: its memory is the graph's."""
    call = make_calls()[name]
    ref = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        wait_inputs(side)
        out = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for x in out:
        x.zero_()
    gr.replay()
    other = call(None)  # nothing of the graph's memory
    gr.replay()
    torch.cuda.synchronize()
    for x, y, r in zip(out, other, ref):
        assert torch.equal(x, r) and torch.equal(y, r)


@pytest.mark.parametrize("split_call", ["prefill", "decode", "decode_pair"])
def test_workspaces_do_not_pile_up(cuda_dev, split_call):
    """Calls one after the other on a stream use one workspace, however long
    the current stream is busy."""
    call = make_calls()[split_call]
    side = torch.cuda.Stream()
    wait_inputs(side)
    active = lambda: torch.cuda.memory_stats()["active_bytes.all.current"]  # noqa: E731
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    keep = [call(side)]
    used = sum(x.nbytes for x in keep[0])
    torch.cuda._sleep(400_000_000)
    start = active()
    for _ in range(8):
        keep.append(call(side))
    grown = active() - start
    torch.cuda.synchronize()
    assert grown <= 8 * (used + 8 * 512), (grown, used)


@pytest.mark.parametrize("given", [False, True])
def test_host_threads(cuda_dev, given):
    """Four host threads, each with a stream of its own, current or given."""
    import threading
    sets = [make_calls() for _ in range(4)]
    refs = [{n: [x.clone() for x in c[n](None)] for n in NAMES} for c in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        try:
            for _ in range(10):
                for n in NAMES:
                    if given:
                        out = sets[i][n](s)
                        torch.cuda.current_stream().wait_stream(s)
                        ok = all(torch.equal(x, r) for x, r in zip(out, refs[i][n]))
                    else:
                        with torch.cuda.stream(s):
                            out = sets[i][n](None)
                            ok = all(torch.equal(x, r) for x, r in zip(out, refs[i][n]))
                    if not ok:
                        wrong.append((i, n))
        except Exception as e:  # noqa: BLE001 - reported below
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
