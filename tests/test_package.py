"""The package's names (CPU)."""


def test_names_follow_the_binding(monkeypatch):
    """What replaces a function of the binding (a wrapper that counts or times
    calls, a stand-in in a test) is what the package gives from then on."""
    import bitlinear_w1_a8_amd as bl
    from bitlinear_w1_a8_amd import binding
    before = bl.forward
    assert before is binding.forward
    stand_in = lambda *args: None  # noqa: E731
    monkeypatch.setattr(binding, "forward", stand_in)
    assert bl.forward is stand_in
    monkeypatch.undo()
    assert bl.forward is before
