"""The delta rule's and the norm's calls without a GPU: what the C ABI and the torch binding refuse on the host, before any
HIP call, with the documented status and a message naming the argument; and the workspace sizes."""
import os

import pytest
import torch

FAKE = 0x10000          # 16-byte aligned, never dereferenced: every call below fails validation
MIS = 0x10008           # 8-byte aligned only


@pytest.fixture(scope="module")
def lib():
    import selective_state_space_14_amd as ssd
    if not os.path.exists(ssd.LIB_PATH):
        from selective_state_space_14_amd import build
        build.build(verbose=False)
    return ssd.load()


def at(i):
    return FAKE + 0x1000 * i


HEAD = dict(B=2, L=100, H=8, P=64, N=64, G=2, chunk=64, dtype=1, q=at(1), qs=128, k=at(2), ks=128, v=at(3), vs=512,
            dt=at(4), dts=8, sp=0, dtb=None, A=at(5), beta=at(6), bs=8, sig=0, scale=0.125, qkn=0)
COMMON = [
    (dict(dtype=2), 3, "dtype=2"),
    (dict(B=-1), 2, "B=-1"),
    (dict(H=0), 2, "H=0"),
    (dict(G=0), 2, "G=0"),
    (dict(H=9), 2, "H=9 is not divisible by G=2"),
    (dict(P=32), 3, "P=32"),
    (dict(P=256), 3, "P=256"),
    (dict(N=16), 3, "N=16"),
    (dict(B=1 << 25), 2, "is too large"),
    (dict(sp=2), 3, "dt_softplus=2"),
    (dict(sig=-1), 3, "beta_sigmoid=-1"),
    (dict(qkn=3), 3, "qk_norm=3"),
    (dict(q=None), 1, "q is NULL"),
    (dict(k=MIS), 4, "k="),
    (dict(v=None), 1, "v is NULL"),
    (dict(dt=None), 1, "dt is NULL"),
    (dict(beta=None), 1, "beta is NULL"),
    (dict(A=None), 1, "A is NULL"),
    (dict(qs=64), 2, "q row stride 64"),
    (dict(ks=0), 2, "k row stride 0"),
    (dict(vs=516), 4, "v row stride 516"),
    (dict(dts=4), 2, "dt / beta row strides (4, 8)"),
    (dict(bs=0), 2, "dt / beta row strides (8, 0)"),
    (dict(vs=(1 << 22) + 8), 2, "above 4194304"),
    (dict(ys=256), 2, "row stride 256"),
    (dict(dt=FAKE + 2), 4, "dt="),
]
SCAN = [
    (dict(L=-1), 2, "L=-1"),
    (dict(L=(1 << 30) + 1), 2, "L=1073741825 is above"),
    (dict(chunk=128), 3, "chunk=128"),
    (dict(h0=MIS), 4, "init_state"),
    (dict(len=FAKE + 2), 4, "lengths"),
    (dict(doc=FAKE + 1), 4, "doc_ids"),
    (dict(ws=None), 5, "smaller than the required"),
    (dict(wsb=1000), 5, "workspace_bytes=1000"),
    (dict(ws=MIS), 4, "workspace="),
]


def head(a, lead):
    return [a[n] for n in lead] + [a[n] for n in ("q", "qs", "k", "ks", "v", "vs", "dt", "dts", "sp", "dtb", "A", "beta", "bs",
                                                  "sig", "scale", "qkn")]


def fwd(lib, over):
    a = dict(HEAD, doc=None, len=None, h0=None, hf=None, y=at(7), ys=512, ws=at(8), wsb=1 << 30)
    a.update(over)
    return lib.ssd_delta_scan_fwd(*head(a, ("B", "L", "H", "P", "N", "G", "chunk", "dtype")), a["doc"], a["len"], a["h0"],
                                  a["hf"], a["y"], a["ys"], a["ws"], a["wsb"], None)


def step(lib, over):
    a = dict(HEAD, state=at(7), y=at(8), ys=512)
    a.update(over)
    return lib.ssd_delta_step(*head(a, ("B", "H", "P", "N", "G", "dtype")), a["state"], a["y"], a["ys"], None)


def bwd(lib, over):
    a = dict(HEAD, doc=None, len=None, h0=None, gy=at(7), ys=512, gS=None, dq=at(8), dqs=128, dk=at(9), dks=128, dv=at(10),
             dvs=512, ddt=at(11), ddts=8, dbeta=at(12), dbs=8, dA=at(13), ddtb=None, dh0=None, ws=at(14), wsb=1 << 30)
    a.update(over)
    return lib.ssd_delta_scan_bwd(*head(a, ("B", "L", "H", "P", "N", "G", "chunk", "dtype")), a["doc"], a["len"], a["h0"],
                                  a["gy"], a["ys"], a["gS"], a["dq"], a["dqs"], a["dk"], a["dks"], a["dv"], a["dvs"],
                                  a["ddt"], a["ddts"], a["dbeta"], a["dbs"], a["dA"], a["ddtb"], a["dh0"], a["ws"], a["wsb"],
                                  None)


def refused(lib, st, status, needle):
    assert st == status, (st, lib.ssd_last_error())
    assert needle in lib.ssd_last_error().decode(), lib.ssd_last_error()


@pytest.mark.parametrize("over,status,needle", COMMON + SCAN + [
    (dict(y=None), 1, "y is NULL"),
    (dict(hf=MIS), 4, "final_state"),
    (dict(y=at(3)), 2, "y must not alias"),
    (dict(y=at(9), hf=at(9)), 2, "y must not alias"),
])
def test_delta_scan_refusals(lib, over, status, needle):
    refused(lib, fwd(lib, over), status, needle)


@pytest.mark.parametrize("over,status,needle", COMMON + [
    (dict(state=None), 1, "state is NULL"),
    (dict(state=MIS), 4, "state="),
    (dict(y=at(7)), 2, "y must not alias"),
    (dict(y=at(1)), 2, "y must not alias"),
])
def test_delta_step_refusals(lib, over, status, needle):
    refused(lib, step(lib, over), status, needle)


@pytest.mark.parametrize("over,status,needle", COMMON + SCAN + [
    (dict(gy=None), 1, "grad_y is NULL"),
    (dict(dq=None), 1, "dq is NULL"),
    (dict(dk=MIS), 4, "dk="),
    (dict(dvs=500), 2, "dv row stride 500"),
    (dict(ddt=None), 1, "ddt is NULL"),
    (dict(dbeta=None), 1, "dbeta is NULL"),
    (dict(ddts=7), 2, "ddt / dbeta row strides (7, 8)"),
    (dict(dqs=1 << 23), 2, "above 4194304"),
    (dict(dA=None), 1, "dA is NULL"),
    (dict(gS=MIS), 4, "grad_final_state"),
    (dict(dh0=MIS), 4, "grad_init_state"),
    (dict(dq=at(1)), 2, "an output must not alias an input"),
    (dict(gS=at(20), dh0=at(20)), 2, "an output must not alias an input"),
    (dict(dq=at(9)), 2, "two outputs must not alias"),
])
def test_delta_bwd_refusals(lib, over, status, needle):
    refused(lib, bwd(lib, over), status, needle)


def norm(lib, bwd, over):
    a = dict(R=10, groups=1, W=64, xd=1, d=1, rms=0, eps=1e-5, x=at(1), xs=64, w=at(2), b=at(3), z=None, zs=0, y=at(4), ys=64,
             gy=at(5), gys=64, dx=at(6), dxs=64, dw=at(7), db=at(8), dz=None, dzs=0, ws=at(9), wsb=1 << 30)
    a.update(over)
    row = [a[n] for n in ("R", "groups", "W", "xd", "d", "rms", "eps", "x", "xs", "w", "b", "z", "zs")]
    if not bwd:
        return lib.ssd_norm_fwd(*row, a["y"], a["ys"], None)
    return lib.ssd_norm_bwd(*row, *(a[n] for n in ("gy", "gys", "dx", "dxs", "dw", "db", "dz", "dzs", "ws", "wsb")), None)


NORM = [
    (dict(xd=2), 3, "dtype=2"),
    (dict(d=-1), 3, "dtype=-1"),
    (dict(R=-1), 2, "R=-1"),
    (dict(groups=0), 2, "groups=0"),
    (dict(R=1 << 30, groups=4), 2, "too many"),
    (dict(W=0), 2, "W=0"),
    (dict(W=16385), 3, "W=16385"),
    (dict(W=8193, xs=8193, ys=8193, gys=8193, dxs=8193), 4, "W=8193 above 8192"),
    (dict(W=16384, xs=16386, ys=16384, gys=16384, dxs=16384), 4, "W=16384 above 8192"),
    (dict(rms=2), 3, "rms=2"),
    (dict(eps=-1.0), 3, "eps=-1"),
    (dict(eps=float("nan")), 3, "eps=nan"),
    (dict(x=None), 1, "x is NULL"),
    (dict(xs=63), 2, "x row stride 63 is smaller"),
    (dict(groups=2), 2, "smaller than the row width 128"),
    (dict(xs=(1 << 22) + 1), 2, "above 4194304"),
    (dict(x=FAKE + 1), 4, "x="),
    (dict(z=at(20), zs=32), 2, "z row stride 32"),
    (dict(w=FAKE + 2), 4, "weight"),
    (dict(b=FAKE + 1), 4, "bias"),
]


@pytest.mark.parametrize("over,status,needle", NORM + [
    (dict(y=None), 1, "y is NULL"),
    (dict(y=at(1)), 2, "y must not alias"),
    (dict(z=at(4), zs=64), 2, "y must not alias"),
])
def test_norm_fwd_refusals(lib, over, status, needle):
    refused(lib, norm(lib, False, over), status, needle)


@pytest.mark.parametrize("over,status,needle", NORM + [
    (dict(gy=None), 1, "grad_y is NULL"),
    (dict(dx=None), 1, "dx is NULL"),
    (dict(dz=at(20), dzs=64), 1, "dz is given but z is NULL"),
    (dict(dx=at(5)), 2, "must not alias"),
    (dict(z=at(20), zs=64, dz=at(6), dzs=64), 2, "must not alias"),
    (dict(dw=FAKE + 2), 4, "dweight"),
    (dict(ws=None), 5, "smaller than the required"),
    (dict(wsb=16), 5, "workspace_bytes=16"),
    (dict(ws=MIS), 4, "workspace="),
])
def test_norm_bwd_refusals(lib, over, status, needle):
    refused(lib, norm(lib, True, over), status, needle)


def test_nothing_to_do_needs_no_gpu(lib):
    assert fwd(lib, dict(B=0)) == 0 and fwd(lib, dict(L=0)) == 0 and step(lib, dict(B=0)) == 0 and bwd(lib, dict(B=0)) == 0
    assert norm(lib, False, dict(R=0)) == 0 and norm(lib, True, dict(R=0, dw=None, db=None)) == 0


def test_workspace_sizes(lib):
    size = lib.ssd_delta_scan_workspace_size
    assert size(0, 100, 8, 64, 64, 2, 1) == 0 and size(2, 0, 8, 64, 64, 2, 1) == 0 and size(2, 100, 0, 64, 64, 2, 1) == 0
    # T (packed), Att, four arrays of scalars and a decay of every chunk and head
    assert size(2, 100, 8, 64, 64, 2, 1) == 32 * (10240 + 6144 + 1024) + 256
    # a long row of few heads: the states and transitions of its superchunks too
    assert size(1, 32768, 16, 128, 128, 16, 1) > 512 * 16 * (10240 + 6144 + 1024 + 4)
    assert size(1, 32768, 16, 128, 128, 16, 0) == 512 * 16 * (10240 + 10240 + 1024 + 4)
    back = lib.ssd_delta_scan_bwd_workspace_size
    assert back(2, 0, 8, 64, 64, 2, 1) == 0
    assert back(2, 100, 8, 64, 64, 2, 1) >= 32 * (3 * 12288 + 9 * 256 + 4 + 4 * 64 * 64 * 4 + 8)
    assert lib.ssd_norm_bwd_workspace_size(0, 1, 64) == 0
    assert lib.ssd_norm_bwd_workspace_size(10, 2, 64) >= 2 * 64 * 4


class TestBinding:
    """The torch binding refuses tensors that the library could not read, naming them (no GPU: tensors off the GPU come
    last in each check, and every call here fails before)."""

    def test_host_tensors(self):
        import selective_state_space_14_amd as ssd
        x = torch.zeros(4, 64)
        for call in (lambda: ssd.ssd_norm_fwd(x), lambda: ssd.ssd_norm_bwd(x, x)):
            with pytest.raises((ValueError, TypeError), match="x"):
                call()
        q, v, h = torch.zeros(2, 10, 128), torch.zeros(2, 10, 512), torch.zeros(2, 10, 8)
        dims = dict(H=8, P=64, N=64, G=2)
        for call in (lambda: ssd.ssd_delta_scan_fwd(q, q, v, h, h[0, 0], h, **dims),
                     lambda: ssd.ssd_delta_scan_bwd(q, q, v, h, h[0, 0], h, v, **dims),
                     lambda: ssd.ssd_delta_step(q[:, 0], q[:, 0], v[:, 0], h[:, 0], h[0, 0], h[:, 0],
                                                torch.zeros(2, 8, 64, 64), **dims)):
            with pytest.raises((ValueError, TypeError), match="q"):
                call()
