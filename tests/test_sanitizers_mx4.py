"""The MX4 and expert entry points' host code (argument checks, plans, sizes) under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_sanitizers.py runs the others (CPU only)."""
import test_sanitizers as san


def test_mx4_host_code_under_asan_ubsan(monkeypatch):
    ran = []
    run = san.run
    monkeypatch.setattr(san, "run", lambda env, preload, tests: ran.append(run(
        env, preload, ["tests/test_mx4.py", "tests/test_mx4_limits.py", "tests/test_mx4_plans.py"])))
    san.test_library_host_code_under_asan_ubsan()
    assert ran
