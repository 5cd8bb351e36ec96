"""The smoke run launches every operator of the library (needs a B200)."""
import pytest

import kda_chunked_recurrent_b200 as K

pytestmark = pytest.mark.gpu


def test_smoke_calls_every_operator(monkeypatch, capsys):
    import __graft_entry__ as entry
    names = ["prefill", "decode", "conv_prefill", "conv_decode", "scan_prefill", "scan_decode",
             "rms_norm"]
    called = set()

    def watch(name):
        fn = getattr(K, name)

        def wrapped(*a, **kw):
            called.add(name)
            return fn(*a, **kw)
        return wrapped

    for name in names:
        monkeypatch.setattr(K, name, watch(name))
    entry.smoke()
    assert called == set(names) and "smoke ok" in capsys.readouterr().out
