"""A block's run of operators as they are used together: norm, routing, pairs sorted by expert, quantised rows, the
experts' two products, collected with their weights, and the norm that closes the block and opens the next.
Each stage is checked in fp64 from the stage before as the GPU computed it, so a bound holds stage by stage."""
import pytest
import torch

import quantized_expert_ffn_gemm_b200 as moe
from tests import block_ref as ref
from tests.block_ref import U32, close, rounded

pytestmark = pytest.mark.gpu

H, E, K, I = 256, 24, 3, 128


class Block:
    def __init__(self, T, seed=0):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s, m=1.0: torch.randn(*s, generator=g) * m  # noqa: E731
        self.T = T
        self.r, self.prev = n(T, H).cuda(), n(T, H, m=0.5).cuda()
        self.Wr, self.pre_gain, self.post_gain = n(E, H, m=0.1).cuda(), (1 + n(H, m=0.1)).cuda(), (1 + n(H, m=0.1)).cuda()
        self.gate = torch.rand(H, generator=g).cuda()
        q = lambda *s: moe.mx4_quantize(n(*s, m=s[-1] ** -0.5).cuda())  # noqa: E731
        self.w_gate, self.w_up, self.w_down = q(E, I, H), q(E, I, H), q(E, H, I)
        self.route_ws = moe.Workspace.for_layer(H, E, K, 64, False, T)
        self.ws = moe.Workspace(moe.block_workspace_bytes(T, K, E, H))

    def forward(self):
        s = {}
        s["r1"], s["u"], s["ry"], s["ru"] = moe.block_norm(self.r, self.prev, post_gain=self.post_gain, gate=self.gate,
                                                           pre_gain=self.pre_gain)
        s["idx"], s["w"] = moe.router_topk(s["u"], self.Wr, None, K, self.route_ws)
        s["plan"] = moe.sort_pairs(s["idx"], E, self.ws)
        s["a"] = moe.mx4_quantize(s["u"], s["plan"]["row_of"], s["plan"]["offsets"])
        s["h"] = moe.mx4_product(s["a"], self.w_gate, s["plan"]["offsets"], up=self.w_up, ws=self.ws)
        s["ha"] = moe.mx4_quantize(s["h"])
        s["o"] = moe.mx4_product(s["ha"], self.w_down, s["plan"]["offsets"], ws=self.ws)
        s["y"] = moe.collect(s["o"], s["plan"]["row_of"], s["w"])
        s["r2"], s["u2"], s["ry2"], s["ru2"] = moe.block_norm(s["r1"], s["y"], post_gain=self.post_gain, gate=self.gate,
                                                              pre_gain=self.pre_gain)
        return s

    def backward(self, s, dr2, du2):
        """Of the closing norm and the way back: to the experts' rows and the routing weights."""
        g = moe.block_norm_backward(dr2, du2, s["r2"], s["ru2"], s["y"], s["ry2"], post_gain=self.post_gain, gate=self.gate,
                                    pre_gain=self.pre_gain, ws=self.ws)
        g["d_rows"], g["d_w"] = moe.collect_backward(g["dy"], s["o"], s["plan"]["row_of"], s["w"], s["plan"]["offsets"])
        g["dx"] = moe.collect(g["d_rows"], s["plan"]["row_of"])
        return g


def tensors(s):
    out = []
    for v in s.values():
        out += list(v.values()) if isinstance(v, dict) else list(v) if isinstance(v, tuple) else [v]
    return [t for t in out if t is not None]


@pytest.mark.parametrize("T", [1, 4, 37, 300])
def test_each_stage_of_a_block(T):
    b = Block(T, T)
    s = b.forward()
    c = lambda t: t.cpu().double()  # noqa: E731
    plan = ref.sort_pairs(s["idx"].cpu(), E)
    for n in plan:
        assert torch.equal(plan[n], s["plan"][n].cpu())
    src = plan["src"].long()
    code, byte = ref.mx4_quantize(c(s["u"]))
    assert torch.equal(ref.pack(code)[src], s["a"].codes.cpu()) and torch.equal(byte[src], s["a"].scales.cpu())
    want, err = ref.mx4_product(ref.mx4_values(s["a"]), ref.mx4_values(b.w_gate), plan["offsets"], ref.mx4_values(b.w_up))
    close(s["h"], want, err + rounded(want, torch.float16), "h")
    code, byte = ref.mx4_quantize(c(s["h"]))
    assert torch.equal(ref.pack(code), s["ha"].codes.cpu()) and torch.equal(byte, s["ha"].scales.cpu())
    want, err = ref.mx4_product(ref.mx4_values(s["ha"]), ref.mx4_values(b.w_down), plan["offsets"])
    close(s["o"], want, err + rounded(want, torch.float16), "o")
    each = ref.spread(plan["row_of"], c(s["o"])) * c(s["w"])[..., None]
    close(s["y"], each.sum(1), (K + 2) * U32 * each.abs().sum(1), "y")
    R, U, _, RU, mag = ref.block_norm(c(s["r1"]), c(s["y"]), c(b.post_gain), c(b.gate), 1.0, c(b.pre_gain))
    close(s["r2"], R, 64 * U32 * mag, "r2")
    g = b.backward(s, torch.randn_like(s["r2"]), torch.randn_like(s["u2"]))
    dy = c(g["dy"])
    want = (c(s["w"])[..., None] * dy[:, None]).view(-1, H)[torch.argsort(plan["row_of"].view(-1))]
    close(g["d_rows"], want, U32 * want.abs() + rounded(want, torch.float16), "d_rows")
    back = ref.spread(plan["row_of"], c(g["d_rows"]))
    close(g["dx"], back.sum(1), (K + 2) * U32 * back.abs().sum(1), "dx")
    for ws in (b.ws, b.route_ws):
        assert moe.read_device_error(ws) == 0


def test_two_blocks_at_once_and_captured():
    """Two blocks on two streams, each with its workspaces; then one captured, replayed on new inputs while the
    other runs: bit for bit what each gives alone."""
    a, b = Block(64, 1), Block(200, 2)
    alone = [tensors(x.forward()) for x in (a, b)]
    alone = [[t.clone() for t in x] for x in alone]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for st, x in zip(streams, (a, b)):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(tensors(x.forward()))
        torch.cuda.synchronize()
        for g, w in zip(got, alone):
            assert all(torch.equal(p, q) for p, q in zip(g, w))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = tensors(a.forward())
    a.r.neg_()
    with torch.cuda.stream(streams[1]):
        beside = tensors(b.forward())
    graph.replay()
    torch.cuda.synchronize()
    again = tensors(a.forward())
    assert all(torch.equal(p, q) for p, q in zip(held, again))
    assert all(torch.equal(p, q) for p, q in zip(beside, alone[1]))
    assert not torch.equal(held[0], alone[0][0])
