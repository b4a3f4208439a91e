"""The operators around int8 experts on the host: the 64-bit references on cases
worked by hand, and the refusals, which come before any launch."""
import numpy as np
import pytest
import torch

import int8_ops_ref as ref
import moe_router_softmax_b200 as moe
from test_abi_host import _null_layer

A, NULL = 256, None  # an aligned address that is never read


def test_reference_routing_by_hand():
    l = np.array([[0.0, 1.0, 1.0, -np.inf, 2.0, np.nan]], np.float32)
    ids, w = ref.route(l, 4)
    assert ids.tolist() == [[4, 1, 2, 0]]  # ties to the lower id
    e = np.exp([2.0, 1.0, 1.0, 0.0])
    assert np.allclose(w[0], e / e.sum(), rtol=1e-15)
    ids, w = ref.route(l, 6, renorm=False, scale=2.0)
    assert ids.tolist() == [[4, 1, 2, 0, -1, -1]] and np.isclose(w.sum(), 2.0)
    # the bias chooses but does not weigh
    b = np.array([0.0, 0.0, 0.0, 9.0, -9.0, 9.0], np.float32)
    ids, w = ref.route(l, 2, bias=b, score="sigmoid", renorm=False)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, 1.0 / (1.0 + np.exp(-1.0)))
    # groups {0,1} {2,3} {4,5}: by their best two, 0.5 + 0.73 against 0.88
    ids, _ = ref.route(l, 2, score="sigmoid", n_group=3, topk_group=1, group_top=2)
    assert ids.tolist() == [[1, 0]]
    ids, _ = ref.route(l, 2, score="sigmoid", n_group=3, topk_group=1, group_top=1)
    assert ids.tolist() == [[4, -1]]
    ids, w = ref.route(np.full((1, 4), -np.inf, np.float32), 2)
    assert ids.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]


def test_reference_codes_and_norm_by_hand():
    q, s = ref.codes(np.array([[127.0, -63.5, 0.5, 0.0], [0.0, 0.0, 0.0, 0.0]]))
    assert q.tolist() == [[127, -64, 0, 0], [0, 0, 0, 0]] and s.tolist() == [1.0, 0.0]
    n, _ = ref.norm(np.array([[3.0, -3.0]]), np.array([1.0, 2.0]), 1e-12, 0.5)
    assert np.allclose(n, [[1.5, -2.5]])


def _refused(st, frag, status=None):
    assert st == (moe.MOE_ERR_INVALID_ARG if status is None else status)
    assert frag in moe.moe_last_error(), moe.moe_last_error()


def test_route_scored_refusals():
    def call(logits=A, T=4, E=8, k=2, score=0, G=1, tg=1, gt=1, scale=1.0, ids=A, w=A):
        return moe._lib.moe_route_scored(logits, NULL, T, E, k, score, G, tg, gt, 1, scale, ids, w, NULL)

    _refused(call(E=0), "E=0")
    _refused(call(E=1025), "E=1025")
    _refused(call(k=9), "k=9")
    _refused(call(E=64, k=33), "k=33")
    _refused(call(T=-1), "T=-1")
    _refused(call(score=2), "score")
    _refused(call(G=3), "n_group=3")
    _refused(call(E=64, G=64), "n_group=64")
    _refused(call(G=4, tg=5), "topk_group=5")
    _refused(call(G=4, tg=0), "topk_group=0")
    _refused(call(G=4, tg=1, k=3), "k=3")
    _refused(call(gt=3), "group_top=3")
    _refused(call(G=8, tg=8, gt=2), "group_top=2")
    _refused(call(scale=float("inf")), "scale")
    _refused(call(scale=float("nan")), "scale")
    _refused(call(logits=NULL), "NULL")
    _refused(call(w=NULL), "NULL")
    assert call(T=0, logits=NULL, ids=NULL, w=NULL) == moe.MOE_OK


def test_linear_refusals():
    def call(xq=A, T=4, N=8, K=64, y=A):
        return moe._lib.moe_linear_int8(xq, A, A, A, T, N, K, y, 0, NULL)

    _refused(call(T=-1), "T=-1")
    _refused(call(N=0), "N=0")
    _refused(call(K=0), "K=0")
    _refused(call(K=24), "K=24")
    _refused(call(K=65552), "K=65552")
    _refused(call(xq=NULL), "NULL")
    _refused(call(y=A + 8), "aligned")
    assert call(T=0, xq=NULL, y=NULL) == moe.MOE_OK


def test_ffn_refusals():
    def call(layer=None, T=4, k=2, xq=A, ws=A, ws_bytes=1 << 30):
        layer = _null_layer(fmt=1) if layer is None else layer
        return moe._lib.moe_grouped_ffn_w8a8(layer, xq, A, T, k, A, A, A, A, ws, ws_bytes, NULL)

    _refused(call(layer=_null_layer(fmt=0)), "int8 experts", moe.MOE_ERR_UNSUPPORTED)
    _refused(call(layer=_null_layer(fmt=2)), "int8 experts", moe.MOE_ERR_UNSUPPORTED)
    _refused(call(layer=_null_layer(fmt=1, H=96)), "H=96")
    _refused(call(layer=_null_layer(fmt=1, slot_table=A, pool=A)), "pool_slots")
    _refused(call(k=9), "k=9")
    _refused(call(T=1 << 30, k=2), "T*k")
    _refused(call(xq=NULL), "NULL")
    _refused(call(xq=A + 8), "aligned")
    _refused(call(ws_bytes=16), "workspace")
    assert call(T=0, xq=NULL, ws=NULL) == moe.MOE_OK
    L = _null_layer(fmt=1)
    need = moe._lib.moe_grouped_ffn_w8a8_workspace(L, 4, 2)
    assert need >= 4 * 2 * 128 * 4 and need % 256 == 0
    assert moe._lib.moe_grouped_ffn_w8a8_workspace(None, 4, 2) == 0


def test_norm_refusals():
    L = moe._lib

    def norm(x=A, wt=A, T=2, H=64, eps=1e-6, off=0.0, xn=A, xq=NULL, sx=NULL):
        return L.moe_norm(x, wt, T, H, eps, off, xn, xq, sx, NULL)

    _refused(norm(H=96), "H=96")
    _refused(norm(H=16448), "H=16448")
    _refused(norm(T=-1), "T=-1")
    _refused(norm(eps=0.0), "eps")
    _refused(norm(eps=float("nan")), "eps")
    _refused(norm(off=float("inf")), "finite")
    _refused(norm(x=NULL), "NULL")
    _refused(norm(wt=NULL), "NULL")
    _refused(norm(xn=NULL), "neither")
    _refused(norm(xq=A), "go together")
    _refused(norm(sx=A), "go together")
    _refused(norm(x=A + 8), "aligned")
    assert norm(T=0, x=NULL, xn=NULL) == moe.MOE_OK  # an empty batch

    def after(z=A, res=A, nw=A, T=2, H=64, y=A, xn=A, xq=NULL, sx=NULL, bs=1.0, gh=NULL):
        return L.moe_residual_norm(z, res, A, gh, NULL, nw, T, H, 1e-6, 0.0, 1.0, bs, y, xn, xq, sx, NULL)

    _refused(after(z=NULL), "NULL")
    _refused(after(res=NULL), "NULL")
    _refused(after(y=NULL), "NULL")
    _refused(after(nw=NULL), "need")
    _refused(after(xn=NULL), "without an output")
    _refused(after(bs=float("nan")), "finite")
    _refused(after(gh=A + 4), "aligned")
    _refused(after(xq=A), "go together")

    def comb(rows=A, pos=A, k=2, T=2):
        return L.moe_combine_norm(rows, pos, A, k, A, A, NULL, NULL, A, T, 64, 1e-6, 0.0, 1.0, 1.0, A, A, NULL, NULL,
                                  NULL)

    _refused(comb(k=0), "k=0")
    _refused(comb(k=33), "k=33")
    _refused(comb(rows=NULL), "NULL")
    _refused(comb(pos=NULL), "NULL")
    _refused(comb(T=1 << 30, k=8), "T*k")
    assert comb(T=0) == moe.MOE_OK


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_norm(x, x[0])
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_route_scored(torch.zeros((2, 8)), 2)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_linear_int8(x.to(torch.int8), x[:, 0].float(), x.to(torch.int8), x[:, 0].float())


class _On:
    """Stands for a CUDA tensor on a device; its memory is never reached."""

    is_cuda, dtype = True, torch.int8

    def __init__(self, dev, *shape):
        self.dev, self.shape, self.device = dev, shape, f"cuda:{dev}"

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.dev


@pytest.mark.parametrize("name", ["home", "pool", "slot_table"])
def test_ffn_refuses_a_layer_on_another_device(name):
    class Layer:
        E, H, I = 4, 64, 64
        home, pool, slot_table = _On(0), _On(0), _On(0)

    setattr(Layer, name, _On(1))
    with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
        moe.moe_grouped_ffn_w8a8(Layer(), _On(0, 2, 64), None, 2, None, None, None)


@pytest.mark.parametrize("E,H,I,k,T,rows", [
    (128, 2816, 704, 8, 1, True), (128, 2816, 704, 8, 5, True), (128, 2816, 704, 8, 6, False),
    (2, 4096, 4096, 1, 1, True), (2, 4096, 4096, 1, 8, False), (2, 4096, 4096, 1, 40, False),
    (4, 4096, 2048, 2, 1, True), (4, 4096, 2048, 2, 4, False), (8, 16384, 16384, 8, 1, True),
    (8, 1024, 512, 2, 8, True), (16, 512, 256, 4, 10, True), (16, 512, 256, 4, 11, False)])
def test_ffn_few_routes_of_few_large_experts(E, H, I, k, T, rows):
    """Few routes read an expert's weights once per route, which pays while routes that share an expert add few bytes:
    the workspace is then the rows of h alone."""
    need = moe._lib.moe_grouped_ffn_w8a8_workspace(_null_layer(fmt=moe.MOE_W_INT8, E=E, H=H, I=I), T, k)
    h = (T * k * I * 4 + 255) // 256 * 256
    assert need == h if rows else need > h
    # a workspace for more tokens serves fewer
    assert need >= moe._lib.moe_grouped_ffn_w8a8_workspace(_null_layer(fmt=moe.MOE_W_INT8, E=E, H=H, I=I), T - 1, k)
