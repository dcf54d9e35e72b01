"""The rotary and attention entry points' host code (argument checks, plans, sizes) under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_sanitizers.py runs the others (CPU only)."""
import test_sanitizers as san


def test_attn_host_code_under_asan_ubsan(monkeypatch):
    ran = []
    run = san.run
    monkeypatch.setattr(san, "run", lambda env, preload, tests: ran.append(run(env, preload, ["tests/test_attn.py"])))
    san.test_library_host_code_under_asan_ubsan()
    assert ran
