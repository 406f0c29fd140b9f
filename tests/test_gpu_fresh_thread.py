"""The first thing a host thread does is a call whose memory is all there: no
earlier call of the thread has made the device's context current to it."""
import threading

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
    """name -> call(stream) into tensors of its own, which it returns."""
    g = torch.Generator("cuda").manual_seed(1)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    f4 = dict(dtype=torch.float32, device="cuda")
    u1 = dict(dtype=torch.uint8, device="cuda")
    T, H, R = 40, 16, 512
    x, w, wkv = normal(g, T, R), normal(g, 256, R), normal(g, H * 256, R)
    q, kv, kp = normal(g, T, H, 192), normal(g, T, H, 256), normal(g, T, 64)
    lat, cu, gs = normal(g, T, H, R), i32([0, T]), i32([0, 1])
    cache, dq = normal(g, 8, 64, 576), normal(g, 4, H, 576)
    cache8, sc = cache.to(torch.float8_e4m3fn), torch.tensor([0.5], device="cuda")
    table, lens = i32([list(range(8))] * 4), i32([512, 300, 0, 65])
    y, k, v, o, y4 = (torch.zeros(*s, **bf) for s in (
        (T, 256), (T, H, 128), (T, H, 128), (T, H, 128), (4, H, R)))
    ql, lse, lse4 = torch.zeros(T, H, R, **bf), torch.zeros(T, H, **f4), torch.zeros(4, H, **f4)
    ws = torch.zeros(mla.mla_decode_shared_workspace_bytes(4, H, 4, 1, R, 152), **u1)
    wd = torch.zeros(max(16, mla.mla_decode_workspace_bytes(4, H, 4, R)), **u1)
    a = (q, kv[..., :128], kv[..., 128:], kp, cu, cu)

    def decode(c, s, scale=None):
        mla.decode(dq, c, table, lens, SCALE, 4, kv_scale=scale, workspace=wd, out=y4, lse=lse4,
                   stream=s)
        return y4, lse4

    def shared(c, s, scale=None):
        mla.decode_shared(dq, c, table, lens, gs4, pre, SCALE, kv_scale=scale, workspace=ws, out=y4,
                          lse=lse4, stream=s)
        return y4, lse4
    gs4, pre, none = i32([0, 4]), i32([64]), i32([0, 0])
    return {
        "linear": lambda s: (mla.linear(x, w, out=y, stream=s),),
        "expand_kv": lambda s: mla.expand_kv(x, wkv, H, k_nope=k, v=v, stream=s),
        "absorb_q": lambda s: (mla.absorb_q(q[..., :128], wkv, out=ql, stream=s),),
        "project_v": lambda s: (mla.project_v(lat, wkv, out=o, stream=s),),
        "prefill": lambda s: mla.prefill(*a, SCALE, out=o, lse=lse, stream=s),
        "prefill_shared": lambda s: mla.prefill_shared(*a, gs, none, SCALE, out=o, lse=lse, stream=s),
        "decode": lambda s: decode(cache, s),
        "decode_e4m3": lambda s: decode(cache8, s, sc),
        "decode_shared": lambda s: shared(cache, s),
        "decode_shared_e4m3": lambda s: shared(cache8, s, sc),
    }


NAMES = ["linear", "expand_kv", "absorb_q", "project_v", "prefill", "prefill_shared", "decode",
         "decode_e4m3", "decode_shared", "decode_shared_e4m3"]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_first_call_of_a_thread(cuda_dev, name, captured):
    call = make_calls()[name]
    out = call(None)
    want = [x.clone() for x in out]
    for x in out:
        x.fill_(7)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            call(s)
        except Exception as e:  # noqa: BLE001 - reported below
            wrong.append(repr(e))

    def run():
        t = threading.Thread(target=work)
        t.start()
        t.join()

    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            s.wait_stream(torch.cuda.current_stream())
            run()
            torch.cuda.current_stream().wait_stream(s)
        assert not wrong
        g.replay()
    else:
        run()
    torch.cuda.synchronize()
    assert not wrong
    for x, r in zip(out, want):
        assert torch.equal(x, r)
