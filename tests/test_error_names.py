"""The names in the errors of the operators on latent caches and of rotations."""
import ctypes

import moe_decode_megakernel_02_gb300 as mk
from test_latent import _attention, _structs
from test_rotary import _args as rotation


def message(rc):
    assert rc == mk.ERR_INVALID_ARG
    return mk.lib().mk_last_error().decode()


def test_errors_name_their_operator():
    L, ref = mk.lib(), ctypes.byref
    for over, name in ((dict(x__data=None), "rotate: x"), (dict(o__data=4097), "rotate: out"), (dict(x__dtype=9), "rotate: ")):
        assert message(L.mk_rotate(ref(rotation(**over)), None)).startswith(name)
    for over, name in ((dict(q__data=None), "latent attend: q"), (dict(r__data=4097), "latent attend: q_rope"),
                       (dict(o__data=None), "latent attend: out")):
        att = _attention(*_structs(**over)[:6])
        assert message(L.mk_latent_attend(ref(att), 4096, 1 << 40, None)).startswith(name)
    p, t, q = _structs(q__data=None)[:3]
    got = message(L.mk_latent_write(ref(p), ref(t), 4096, None, 1, ref(q), None, 0, 1e-6, None, None, None))
    assert got.startswith("latent: rows")
