"""What the int8 operators and the balance loss refuse, and where they may run."""
import re

import numpy as np
import pytest
import torch

from quantized_moe_amd import lib
from test_int8 import make_codes, make_scales

gpu = pytest.mark.gpu
DEV = "cuda:0"
P = 1 << 40  # a pointer that is never dereferenced: every call with it is refused
INVALID, UNSUPPORTED, WORKSPACE = lib.MOE_ERR_INVALID_ARG, lib.MOE_ERR_UNSUPPORTED, lib.MOE_ERR_WORKSPACE


class _NoStream:
    cuda_stream = None


def refused(rc, status, message):
    assert rc == status
    assert re.search(message, lib.last_error()), lib.last_error()


def changed(args, **at):
    a = list(args)
    for i, v in at.items():
        a[int(i[1:])] = v
    return a


def test_quantize_refusals():
    f = lib.lib().moe_int8_quantize
    args = (P, 0, 256, 3, 256, P, 256, P, None)
    for at, status, message in ((dict(_3=-1), INVALID, "M -1"), (dict(_3=(1 << 20) + 1), INVALID, "M 1048577"), (dict(_4=24), INVALID, "K 24"),
                                (dict(_4=16400), INVALID, "K 16400"), (dict(_1=2), UNSUPPORTED, "dtype"), (dict(_2=255), INVALID, "ldx 255"),
                                (dict(_2=258), INVALID, "ldx 258"), (dict(_1=1, _2=260), INVALID, "ldx 260"), (dict(_6=264), INVALID, "ldq 264"),
                                (dict(_6=240), INVALID, "ldq 240"), (dict(_0=None), INVALID, "x is null"), (dict(_0=P + 8), INVALID, "x is not 16"),
                                (dict(_5=None), INVALID, "q is null"), (dict(_7=P + 4), INVALID, "s is not 16")):
        refused(f(*changed(args, **at)), status, message)
    assert f(*changed(args, _0=None, _3=0)) == lib.MOE_OK


def test_matmul_refusals():
    f = lib.lib().moe_int8_matmul
    args = (P, 256, P, 3, P, P, 64, 256, P, 0, 64, None, 0, None)
    for at, status, message in ((dict(_3=-1), INVALID, "M -1"), (dict(_7=250), INVALID, "K 250"), (dict(_6=0), INVALID, "N 0"),
                                (dict(_6=65537), INVALID, "N 65537"), (dict(_9=7), UNSUPPORTED, "dtype 7"), (dict(_1=240), INVALID, "ldx 240"),
                                (dict(_1=264), INVALID, "ldx 264"), (dict(_1=(1 << 22) + 16), INVALID, "ldx"), (dict(_10=63), INVALID, "ldy 63"),
                                (dict(_0=None), INVALID, "xq is null"), (dict(_4=P + 8), INVALID, "wq is not"), (dict(_5=None), INVALID, "ws is null"),
                                (dict(_2=P + 4), INVALID, "xs is not"), (dict(_8=None), INVALID, "y is null")):
        refused(f(*changed(args, **at)), status, message)
    assert f(*changed(args, _0=None, _3=0)) == lib.MOE_OK
    for M, N, K in ((33, 64, 16384), (1, 256, 8208), (100, 300, 16384)):
        need = lib.int8_matmul_workspace_bytes(M, N, K)
        assert need == 4 * 4 * M * N
        call = changed(args, _1=K, _3=M, _6=N, _7=K, _10=N)
        refused(f(*changed(call, _11=P, _12=need - 1)), WORKSPACE, "need %d" % need)
        refused(f(*changed(call, _11=None, _12=need)), INVALID, "workspace is null")
    for M, N, K in ((33, 64, 8192), (1, 8192, 16384), (4096, 4096, 16384)):
        assert lib.int8_matmul_workspace_bytes(M, N, K) == 0
    with pytest.raises(lib.MoeError, match="K 17"):
        lib.int8_matmul_workspace_bytes(4, 64, 17)


def test_experts_refusals():
    f = lib.lib().moe_int8_gateup
    args = (P, P, 3, 2, P, P, 8, P, P, P, P, 128, 256, P, 0, None)
    for at, status, message in ((dict(_2=-1), INVALID, "T -1"), (dict(_2=65537), INVALID, "T 65537"), (dict(_3=0), INVALID, "top_k 0"),
                                (dict(_3=9), INVALID, "top_k 9"), (dict(_6=0), INVALID, "n_experts 0"), (dict(_6=1025), INVALID, "n_experts"),
                                (dict(_11=100), INVALID, "f 100"), (dict(_12=8), INVALID, "d 8"), (dict(_14=3), UNSUPPORTED, "dtype 3"),
                                (dict(_13=P + 8), INVALID, "h is not"), (dict(_4=None), INVALID, "offsets is null"), (dict(_10=None), INVALID, "s_up is null")):
        refused(f(*changed(args, **at)), status, message)
    assert f(*changed(args, _0=None, _2=0)) == lib.MOE_OK
    g = lib.lib().moe_int8_down
    need = lib.int8_down_workspace_bytes(3, 2, 256)
    assert need == 3 * 2 * 256 * 4 and lib.int8_down_workspace_bytes(2, 2, 256) == 0
    args = (P, P, 3, 2, P, P, P, 8, P, P, 256, 128, None, P, P, need, None)
    for at, status, message in ((dict(_2=-1), INVALID, "T -1"), (dict(_3=17), INVALID, "top_k 17"), (dict(_10=264), INVALID, "d 264"),
                                (dict(_12=P + 4), INVALID, "add is not"), (dict(_15=need - 1), WORKSPACE, "need"), (dict(_14=None), INVALID, "workspace is null"),
                                (dict(_4=None), INVALID, "wt is null"), (dict(_13=P + 8), INVALID, "y is not")):
        refused(g(*changed(args, **at)), status, message)
    assert g(*changed(args, _0=None, _2=0)) == lib.MOE_OK


def test_balance_refusals():
    f = lib.lib().moe_balance_loss
    need = lib.balance_loss_workspace_bytes(300, 2, 8)
    assert need == 300 * 8 and lib.balance_loss_workspace_bytes(128, 2, 8) == 0
    args = (P, 0, 8, 300, 8, P, 2, 0, 1.0, P, 2, P, P, P, P, need, None)
    for at, status, message in ((dict(_3=-1), INVALID, "T -1"), (dict(_3=65537), INVALID, "T 65537"), (dict(_4=0), INVALID, "n_experts 0"),
                                (dict(_4=1025), INVALID, "n_experts 1025"), (dict(_6=0), INVALID, "top_k 0"), (dict(_6=9), INVALID, "top_k 9"),
                                (dict(_7=2), UNSUPPORTED, "score 2"), (dict(_8=float("inf")), INVALID, "alpha"), (dict(_8=float("nan")), INVALID, "alpha"),
                                (dict(_9=None), INVALID, "2 sequences without"), (dict(_10=0), INVALID, "0 sequences"), (dict(_10=65537), INVALID, "65537 sequences"),
                                (dict(_1=5), UNSUPPORTED, "dtype"), (dict(_2=7), INVALID, "z_stride 7"), (dict(_0=None), INVALID, "z is null"),
                                (dict(_0=P + 2), INVALID, "z is not aligned"), (dict(_1=1, _0=P + 1), INVALID, "z is not aligned"), (dict(_5=None), INVALID, "idx is null"),
                                (dict(_11=P + 2), INVALID, "counts is not 4"), (dict(_13=None), INVALID, "loss is null"), (dict(_15=need - 1), WORKSPACE, "need %d" % need),
                                (dict(_14=P + 8), INVALID, "workspace is not 16")):
        refused(f(*changed(args, **at)), status, message)
    g = lib.lib().moe_balance_loss_backward
    args = (P, 0, 8, 300, 8, P, 2, 0, 1.0, P, 2, P, P, P, P, 8, None)
    for at, status, message in ((dict(_15=7), INVALID, "dz_stride 7"), (dict(_14=None), INVALID, "z or dz is null"), (dict(_14=P + 2), INVALID, "not aligned"),
                                (dict(_13=P + 1), INVALID, "grad_loss is not"), (dict(_12=None), INVALID, "tokens is null"), (dict(_9=None), INVALID, "without")):
        refused(g(*changed(args, **at)), status, message)
    assert g(*changed(args, _3=0)) == lib.MOE_OK


def make_calls(dev, dtype=torch.float32):
    """(name, call(stream), the tensors by name) of every operator on small tensors."""
    def f(*n):
        return torch.zeros(*n, device=dev, dtype=dtype)

    def i8(*n):
        return torch.zeros(*n, dtype=torch.int8, device=dev)

    def i32(*n):
        return torch.zeros(*n, dtype=torch.int32, device=dev)

    w, s = i8(8, 128, 256), f(8, 128)
    return {
        "int8_quantize": (lib.int8_quantize, dict(x=f(4, 256), q=i8(4, 256), s=f(4))),
        "int8_matmul": (lib.int8_matmul, dict(xq=i8(4, 256), xs=f(4), wq=w[0], ws=s[0], y=f(4, 128))),
        "int8_gateup": (lib.int8_gateup, dict(xq=i8(4, 256), xs=f(4), k=2, offsets=i32(9), perm=i32(8), w_gate=w, s_gate=s, w_up=w,
                                              s_up=s, h=f(8, 128))),
        "int8_down": (lib.int8_down, dict(hq=i8(8, 128), hs=f(8), wt=f(4, 2), offsets=i32(9), pos=i32(8), w_down=i8(8, 256, 128),
                                          s_down=f(8, 256), y=f(4, 256), workspace=torch.zeros(4 * 2 * 256 * 4, dtype=torch.uint8, device=dev),
                                          add=f(4, 256))),
        "balance_loss": (lib.balance_loss, dict(z=f(4, 8), idx=i32(4, 2), counts=i32(2, 8), tokens=i32(2), loss=f(2),
                                                workspace=torch.zeros(256, dtype=torch.uint8, device=dev), starts=i32(3))),
        "balance_loss_backward": (lib.balance_loss_backward, dict(z=f(4, 8), idx=i32(4, 2), counts=i32(2, 8), tokens=i32(2),
                                                                  grad_loss=f(2), dz=f(4, 8), starts=i32(3))),
    }


@pytest.mark.parametrize("name", list(make_calls("cpu")))
def test_host_memory_is_refused(name):
    call, args = make_calls("cpu")[name]
    with pytest.raises(ValueError, match="GPU memory"):
        call(**args, stream=_NoStream)


@pytest.mark.parametrize("name", list(make_calls("cpu")))
def test_wrong_types_and_shapes_are_named(name):
    """Every tensor of every call: another type, another shape, gaps."""
    call, args = make_calls("cpu")[name]
    for n, t in args.items():
        if not isinstance(t, torch.Tensor) or n == "workspace":
            continue
        for other in (t.to(torch.float64), torch.cat([t, t], dim=-1), t.repeat_interleave(2, dim=-1)[..., ::2]):
            if n == "idx" and other.dtype == torch.int32 and other.is_contiguous():
                continue  # (more routes a token)
            with pytest.raises((TypeError, ValueError)) as e:
                call(**{**args, n: other}, stream=_NoStream)
            assert name in str(e.value) and "GPU memory" not in str(e.value)


def test_scores_are_named():
    call, args = make_calls("cpu")["balance_loss"]
    with pytest.raises(KeyError):
        call(**args, score="max", stream=_NoStream)


@gpu
@pytest.mark.parametrize("name", list(make_calls("cpu")))
def test_streams(name):
    """A stream of this device is used, one of another is refused."""
    class Elsewhere:  # (its handle is this device's default stream: the call would run)
        cuda_stream = 0
        device_index = 1

    call, args = make_calls(DEV)[name]
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="current device, cuda:0"):
        call(**args, stream=Elsewhere)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(**args, stream=side)
    torch.cuda.synchronize()
    call(**args)
    torch.cuda.synchronize()


@gpu
def test_calls_on_two_streams_at_once():
    """Two products and two losses in flight together, each with its own workspace: the results are those of one at a time."""
    rng = np.random.default_rng(11)
    M, N, K = 60, 256, 16384
    w, ws = torch.from_numpy(make_codes(rng, N, K)).to(DEV), torch.from_numpy(make_scales(rng, 0.05, N)).to(DEV)
    sets = []
    for i in range(2):
        x, xs = torch.from_numpy(make_codes(rng, M, K)).to(DEV), torch.from_numpy(make_scales(rng, 1.0, M)).to(DEV)
        z = torch.from_numpy(rng.standard_normal((3000, 64)).astype(np.float32)).to(DEV)
        idx = z.topk(4, dim=1).indices.to(torch.int32)
        sets.append(dict(x=x, xs=xs, z=z, idx=idx, y=torch.empty(M, N, device=DEV),
                         work=torch.empty(lib.int8_matmul_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV),
                         c=torch.empty(1, 64, dtype=torch.int32, device=DEV), n=torch.empty(1, dtype=torch.int32, device=DEV),
                         loss=torch.empty(1, device=DEV), bw=torch.empty(lib.balance_loss_workspace_bytes(3000, 1, 64), dtype=torch.uint8, device=DEV)))

    def go(s, stream=None):
        lib.int8_matmul(s["x"], s["xs"], w, ws, s["y"], s["work"], stream=stream)
        lib.balance_loss(s["z"], s["idx"], s["c"], s["n"], s["loss"], s["bw"], stream=stream)
    want = []
    for s in sets:
        go(s)
        torch.cuda.synchronize()
        want.append([s[n].clone() for n in ("y", "c", "n", "loss")])
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for s, st in zip(sets, streams):
            go(s, st)
    torch.cuda.synchronize()
    for s, old in zip(sets, want):
        assert all(torch.equal(s[n], o) for n, o in zip(("y", "c", "n", "loss"), old))


@gpu
def test_split_product_in_graphs_that_share_a_workspace():
    """Two captured products over one workspace, replayed in turn on one stream with eager calls between."""
    rng = np.random.default_rng(12)
    M, N, K = 40, 130, 12304
    w, ws = torch.from_numpy(make_codes(rng, N, K)).to(DEV), torch.from_numpy(make_scales(rng, 0.05, N)).to(DEV)
    need = lib.int8_matmul_workspace_bytes(M, N, K)
    assert need > 0
    work = torch.empty(need, dtype=torch.uint8, device=DEV)
    xs = [(torch.from_numpy(make_codes(rng, M, K)).to(DEV), torch.from_numpy(make_scales(rng, 1.0, M)).to(DEV)) for _ in range(2)]
    ys = [torch.empty(M, N, device=DEV) for _ in range(2)]
    want, graphs = [], []
    for (x, s), y in zip(xs, ys):
        lib.int8_matmul(x, s, w, ws, y, work)
        torch.cuda.synchronize()
        want.append(y.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.int8_matmul(x, s, w, ws, y, work)
        graphs.append(g)
    for _ in range(3):
        for g, y, o, (x, s) in zip(graphs, ys, want, xs):
            y.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, o)
            lib.int8_matmul(x, s, w, ws, y, work)
            torch.cuda.synchronize()
            assert torch.equal(y, o)


@gpu
def test_every_launch_is_timed_under_its_name():
    def names(call, **args):
        call(**args)
        lib.profile_reset()
        lib.profile_enable(True)
        try:
            call(**args)
            torch.cuda.synchronize()
            got = lib.profile_collect()
        finally:
            lib.profile_enable(False)
            lib.profile_reset()
        assert all(k == 1 and ms > 0 for k, ms in got.values())
        return sorted(got)
    calls = make_calls(DEV)
    want = {"int8_quantize": ["i8_quantize"], "int8_matmul": ["i8_matmul"], "int8_gateup": ["i8_gateup"], "int8_down": ["i8_combine", "i8_down"],
            "balance_loss": ["balance_small"], "balance_loss_backward": ["balance_backward"]}
    for n, (call, args) in calls.items():
        assert names(call, **args) == want[n]
    for T, more in ((500, []), (1500, ["balance_clear"])):
        big = dict(calls["balance_loss"][1], z=torch.zeros(T, 8, device=DEV), idx=torch.zeros(T, 2, dtype=torch.int32, device=DEV),
                   workspace=torch.empty(8 * T, dtype=torch.uint8, device=DEV))
        assert names(lib.balance_loss, **big) == more + ["balance_count", "balance_forward", "balance_sum"]
    x, w = torch.zeros(33, 16384, dtype=torch.int8, device=DEV), torch.zeros(64, 16384, dtype=torch.int8, device=DEV)
    work = torch.empty(lib.int8_matmul_workspace_bytes(33, 64, 16384), dtype=torch.uint8, device=DEV)
    assert names(lib.int8_matmul, xq=x, xs=torch.zeros(33, device=DEV), wq=w, ws=torch.zeros(64, device=DEV),
                 y=torch.zeros(33, 64, device=DEV), workspace=work) == ["i8_matmul", "i8_matmul_sum"]
