"""moe_block refuses outputs that reach into what it reads (host only: nothing is launched)."""
import pytest

import routed_expert_ffn_05_b200 as M
from test_fp8_host import A, B, C, D, E, F, G, refused

T, d, Fs = 4, 256, 512
H, I, J, K, L = (A + (i << 40) for i in range(1, 6))


def block(x=A, res=B, nw=C, rout=None, tok=None, y=D, ws=E, w1=F, w3=G, w2=H, wr=I, bias=None, route=0, shared=None):
    dims = M.make_dims(T, d, 256, 8, 2, route=route, d_ff_shared=Fs)
    sh = M.make_fp8_ffn_weights(*(shared or [J + (i << 24) for i in range(6)]))
    M.moe_block(dims, M.make_weights(w1, w3, w2, w_router=wr, router_bias=bias), M.make_norm(T, d), sh, x, res, nw, rout, tok,
                y, ws, stream=0)


ROUTED = M.moe_packed_size(M.make_dims(T, d, 256, 8, 2), M.MOE_MAT_W1)


@pytest.mark.parametrize("out", ["y", "ws", "rout"])
@pytest.mark.parametrize("at", [F, F + ROUTED - 256, G + 256, H + ROUTED - 256, I, I + 8 * d * 2 - 16, K, J, J + (1 << 24), J + (5 << 24),
                                J + Fs * d - 256])
def test_an_output_in_the_weights(out, at):
    refused(lambda: block(bias=K, **{out: at // 256 * 256}))


@pytest.mark.parametrize("out", ["y", "ws", "rout"])
def test_an_output_in_the_token_ids(out):
    refused(lambda: block(route=1, wr=None, tok=L, **{out: L}))


@pytest.mark.parametrize("kw", [dict(rout=D), dict(rout=E), dict(y=E), dict(rout=D + T * d * 4 - 2), dict(rout=A), dict(rout=C),
                                dict(rout=B + 2)])
def test_outputs_in_one_another_and_in_the_norms_inputs(kw):
    refused(lambda: block(**kw))
