"""The latent calls without a GPU: the C entries and the binding reject bad
arguments before touching CUDA."""
import ctypes

import pytest
import torch

import fp8_mqa_logits_03_b200 as fx
from fp8_mqa_logits_03_b200 import build

FAKE = ctypes.c_void_p(4096)     # never dereferenced: validation fails first
MIS8 = ctypes.c_void_p(4096 + 8)
MIS4 = ctypes.c_void_p(4096 + 4)
MIS2 = ctypes.c_void_p(4096 + 2)


@pytest.fixture(scope="module")
def L():
    build.build()
    return fx.lib()


def _store(L, c=FAKE, cs=576, pe=FAKE, ps=576, T=4, pos=FAKE, tab=FAKE, maxp=100, slot=FAKE, slots=64, kv=FAKE, s=None,
           ppe=None, q=None, qs=(64, 64), o=None, os_=(64, 64), H=1):
    return L.fp8idx_latent_store(c, cs, pe, ps, T, pos, tab, maxp, 1, slot, slots, kv, s, ppe, q, *qs, o, *os_, H, None)


def test_store_rejects(L):
    assert _store(L, T=-1) == fx.EINVAL
    assert _store(L, maxp=-1) == fx.EINVAL
    assert _store(L, slots=-1) == fx.EINVAL
    assert _store(L, c=None) == fx.EINVAL
    assert _store(L, kv=None) == fx.EINVAL
    assert _store(L, c=MIS8) == fx.EINVAL
    assert b"16-byte" in L.fp8idx_last_error()
    assert _store(L, cs=577) == fx.EINVAL               # a row stride that is no whole 16 bytes
    assert _store(L, tab=MIS8) == fx.EINVAL
    assert _store(L, slot=MIS4) == fx.EINVAL
    assert _store(L, s=FAKE) == fx.EINVAL               # scales without rotated parts
    assert _store(L, ppe=FAKE) == fx.EINVAL
    assert _store(L, q=FAKE) == fx.EINVAL               # q_pe without q_out
    assert _store(L, q=FAKE, o=FAKE, H=0) == fx.EUNSUPPORTED
    assert _store(L, q=FAKE, o=FAKE, H=129) == fx.EUNSUPPORTED
    assert _store(L, q=FAKE, o=MIS8) == fx.EINVAL
    assert _store(L, q=FAKE, o=FAKE, qs=(64, 60)) == fx.EINVAL
    assert _store(L, T=0) == fx.OK
    assert L.fp8idx_last_error() == b""


@pytest.mark.parametrize("T,H,strides", [(4, 1, (0, 64)), (4, 1, (56, 64)), (1, 4, (64, 56)), (1, 4, (64, 0)), (4, 4, (64, 64)),
                                         (4, 4, (248, 64)), (10, 4, (120, 1136)), (4, 3, (200, 72))])
def test_store_rejects_overlapping_output_rows(L, T, H, strides):
    assert _store(L, q=FAKE, o=FAKE, T=T, H=H, os_=strides) == fx.EINVAL
    assert b"overlap" in L.fp8idx_last_error()


def _sparse(L, q=FAKE, qs=(576, 576), kv=FAKE, s=None, pe=None, n=64, slots=FAKE, ld=16, rows=2, topk=16, H=4,
            latent=512, rope=64, scale=0.1, out=FAKE, lse=None, ws=FAKE, nb=1 << 30):
    return L.fp8idx_sparse_latent_attention(q, *qs, kv, s, pe, n, slots, ld, rows, topk, H, latent, rope, scale, out,
                                            lse, ws, nb, None)


def test_sparse_rejects(L):
    assert _sparse(L, H=0) == fx.EUNSUPPORTED
    assert _sparse(L, H=129) == fx.EUNSUPPORTED
    assert _sparse(L, latent=256) == fx.EUNSUPPORTED
    assert _sparse(L, rope=32) == fx.EUNSUPPORTED
    assert _sparse(L, rows=-1) == fx.EINVAL
    assert _sparse(L, topk=-1) == fx.EINVAL
    assert _sparse(L, ld=15) == fx.EINVAL
    assert _sparse(L, n=1 << 31) == fx.EINVAL
    assert _sparse(L, rows=1 << 25, topk=1 << 16, ld=1 << 16) == fx.EINVAL
    assert _sparse(L, q=None) == fx.EINVAL
    assert _sparse(L, slots=None) == fx.EINVAL
    assert _sparse(L, out=None) == fx.EINVAL
    assert _sparse(L, kv=None) == fx.EINVAL
    assert _sparse(L, q=MIS8) == fx.EINVAL
    assert _sparse(L, qs=(576, 572)) == fx.EINVAL
    assert _sparse(L, kv=MIS8) == fx.EINVAL
    assert _sparse(L, out=MIS8) == fx.EINVAL
    assert _sparse(L, slots=MIS2) == fx.EINVAL
    assert _sparse(L, lse=MIS2) == fx.EINVAL
    assert _sparse(L, s=FAKE) == fx.EINVAL
    for scale in (0.0, -0.1, float("nan"), float("inf")):
        assert _sparse(L, scale=scale) == fx.EINVAL
    assert _sparse(L, rows=0) == fx.OK


def _paged(L, q=FAKE, kv=FAKE, s=None, pe=None, bt=FAKE, sl=FAKE, B=2, R=2, mb=4, pages=8, page=64, H=4, latent=512,
           rope=64, out=FAKE, lse=None):
    return L.fp8idx_paged_latent_attention(q, 576, 576, kv, s, pe, bt, sl, B, R, mb, pages, page, H, latent, rope, 0.1,
                                           out, lse, FAKE, 1 << 30, None)


def test_paged_rejects(L):
    assert _paged(L, R=0) == fx.EUNSUPPORTED
    assert _paged(L, R=9) == fx.EUNSUPPORTED
    assert _paged(L, page=32) == fx.EUNSUPPORTED
    assert _paged(L, H=129) == fx.EUNSUPPORTED
    assert _paged(L, latent=128) == fx.EUNSUPPORTED
    assert _paged(L, mb=0) == fx.EINVAL
    assert _paged(L, pages=1 << 25) == fx.EINVAL
    assert _paged(L, B=1 << 24, mb=1 << 10) == fx.EINVAL
    assert _paged(L, B=-1) == fx.EINVAL
    assert _paged(L, bt=None) == fx.EINVAL
    assert _paged(L, sl=MIS2) == fx.EINVAL
    assert _paged(L, pe=FAKE) == fx.EINVAL
    assert _paged(L, B=0) == fx.OK


def test_workspace_queries_reject(L):
    assert L.fp8idx_sparse_latent_attention_workspace(-1, 4, 16) == 0
    assert L.fp8idx_sparse_latent_attention_workspace(1, 0, 16) == 0
    assert L.fp8idx_sparse_latent_attention_workspace(1, 4, -1) == 0
    assert L.fp8idx_paged_latent_attention_workspace(1, 9, 4, 4) == 0
    assert L.fp8idx_paged_latent_attention_workspace(1, 1, 0, 4) == 0
    assert L.fp8idx_paged_latent_attention_workspace(1, 1, 4, 129) == 0


def test_binding_rejects_host_tensors():
    q, kv = torch.zeros(2, 4, 576, dtype=torch.bfloat16), torch.zeros(1, 64, 576, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        fx.sparse_latent_attention(q, kv, torch.zeros(2, 8, dtype=torch.int32), 0.1)
    with pytest.raises(TypeError, match="CUDA"):
        fx.paged_latent_attention(q, kv, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 1, 0.1)
    with pytest.raises(TypeError, match="CUDA"):
        fx.latent_store(q[:, 0, :512], q[:, 0, 512:], torch.zeros(2, dtype=torch.int64), torch.zeros(4, 64),
                        torch.zeros(2, dtype=torch.int64), kv)
    with pytest.raises(TypeError, match="CUDA"):
        fx.sparse_latent_attention(None, kv, None, 0.1)
    with pytest.raises(ValueError, match="both"):
        fx.latent_store(q[:, 0, :512], q[:, 0, 512:], torch.zeros(2, dtype=torch.int64), torch.zeros(4, 64),
                        torch.zeros(2, dtype=torch.int64), kv, s_pages=torch.zeros(1, 64))


@pytest.mark.parametrize("B,R,mb", [(1 << 61, 8, 8), (1 << 62, 4, 4), (1 << 61, 8, 1 << 20), ((1 << 25) // 8 + 1, 8, 1), (1 << 62, 1, 1),
                                    ((1 << 63) - 1, 8, (1 << 31) - 1)])
def test_paged_rejects_sizes_whose_products_overflow(L, B, R, mb):
    assert _paged(L, B=B, R=R, mb=mb) == fx.EINVAL
    assert b"too large" in L.fp8idx_last_error()
    assert L.fp8idx_paged_latent_attention_workspace(B, R, mb, 4) == 0


@pytest.mark.parametrize("rows,topk", [(1 << 62, 16), ((1 << 63) - 1, (1 << 31) - 1), ((1 << 25) + 1, 1), (1, (1 << 24) + 1), (1 << 25, 1 << 16)])
def test_sparse_rejects_sizes_whose_products_overflow(L, rows, topk):
    assert _sparse(L, rows=rows, topk=topk, ld=topk) == fx.EINVAL
    assert b"too large" in L.fp8idx_last_error()
    assert L.fp8idx_sparse_latent_attention_workspace(rows, 4, topk) == 0


def test_binding_belongs_to_one_interpreter_and_torch(L, monkeypatch):
    """A binding that another torch or Python built is neither loaded nor taken as up to date."""
    import sysconfig
    assert not build._stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0.0")
        m.setattr(fx, "_bind_module", None)
        assert build._stale()
        with pytest.raises(RuntimeError, match="build it"):
            fx._bind()
    with monkeypatch.context() as m:
        of = sysconfig.get_config_var
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-30-other" if name == "SOABI" else of(name))
        m.setattr(fx, "_bind_module", None)
        assert build._stale()
        with pytest.raises(RuntimeError, match="build it"):
            fx._bind()
    assert not build._stale()


def test_build_script_is_a_dependency(L, monkeypatch):
    """Other compiler flags mean another library and another binding."""
    import os
    seen = []
    monkeypatch.setattr(build, "_newer", lambda target, deps: seen.append([os.path.abspath(d) for d in deps]) or False)
    build._stale()
    assert len(seen) == 2 and all(os.path.abspath(build.__file__) in deps for deps in seen)
